// Norms of queries and keys for each head with the rotation in the same pass, and
// their gradient.
//
// Forward, for a head x of d elements: r = 1 / sqrt(mean x^2 + eps), n = x r w
// (w: the gains of the queries or of the keys, or 1), y = n with its first R elements
// turned by the row's position, as rope_rotate turns them. Everything between the
// load and the store is FP32, so y is rounded once.
// Backward, for y's gradient: g = the gradient turned back, dw = sum over heads
// and rows of g x r, dx = r (g w - x r mean(g w x r)): what the norm takes out
// of g along x. x r and the mean are worked out again from x, which is read anyway, so
// nothing is kept from the forward pass.
//
// Both read and write each tensor once and are bound by memory, as long as the vector
// unit keeps up: of a wave's 64 lanes it needs about 5 operations an element. A
// head belongs to a group of lanes, two runs of 16 bytes a lane (in the half layout the
// two that turn with each other), so that what a head costs once (the sum's exchanges, 1
// / sqrt) is shared by 16 elements, and several heads of one row go to a group, with
// the row's part of the table and the gains in registers.
// The gains' gradients: a lane keeps the sums of its own elements over all heads of its
// group, a workgroup adds its groups in LDS, and a second launch adds the workgroups' sums
// in one fixed order (no atomics: the same bits every time).
#include <type_traits>

#include "../../include/nrc.h"
#include "div.h"
#include "draft_ops.h"
#include "element.h"

namespace nrc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHead = 256;

struct Part {
    const void* x;
    const void* g;  // backward: y's gradient
    void* out;      // y, or x's gradient
    const void* w;
    int64_t x_rs, x_hs, g_rs, g_hs, out_rs, out_hs;
    int32_t w_type;
    uint32_t heads, units;  // of a row: its heads, and the groups of lanes that they go to
    Div per_row;            // by units
};
struct Dims {
    int64_t T, max_position;
    const int64_t* positions;
    const void* table;
    int32_t d, R;
    uint32_t lanes, shift;  // of a head, and the log of it
    float inv_d, eps;
    bool pass;  // rows without a table row are copied
};

template <int N>
__device__ __forceinline__ void load_gains(const void* w, int32_t type, int32_t e, float (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = type == NRC_DTYPE_F32  ? static_cast<const float*>(w)[e]
               : type == NRC_DTYPE_F16 ? F16::load(static_cast<const _Float16*>(w)[e])
                                       : Bf16::load(static_cast<const uint16_t*>(w)[e]);
    } else {
        if (type == NRC_DTYPE_F32) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                float q[4];
                F32::unpack(load16(static_cast<const float*>(w) + e + i), q);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[i + k] = q[k];
            }
        } else if constexpr (N == 8) {
            const U32x4 v = load16(static_cast<const uint16_t*>(w) + e);
            type == NRC_DTYPE_F16 ? F16::unpack(v, f) : Bf16::unpack(v, f);
        } else {  // 4 gains of 2 bytes
            const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + e);
            float q[8];
            const U32x4 both{v.x, v.y, 0u, 0u};
            type == NRC_DTYPE_F16 ? F16::unpack(both, q) : Bf16::unpack(both, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = q[k];
        }
    }
}

// The sum over a head's lanes, in each of them.
__device__ __forceinline__ float over_lanes(float v, uint32_t lanes) {
    if (lanes > 1) v += lane_xor<1>(v);
    if (lanes > 2) v += lane_xor<2>(v);
    if (lanes > 4) v += lane_xor<4>(v);
    if (lanes > 8) v += lane_xor<8>(v);
    if (lanes > 16) v += lane_xor<16>(v);
    if (lanes > 32) v += lane_xor<32>(v);
    return v;
}

// 1 / sqrt by the hardware's instruction (one step of FP32 off); it takes subnormals for 0, so small ones are scaled.
__device__ __forceinline__ float rsqrt_hw(float v) {
    const bool small = v < 0x1p-100f;
    return __builtin_amdgcn_rsqf(small ? v * 0x1p60f : v) * (small ? 0x1p30f : 1.0f);
}

// A lane's elements of a head, C runs of N: pairs side by side (interleaved: two runs), or run 1 the partners of run 0's
// (half), with the elements that do not turn in two more runs where there are any (REST).
template <int N, bool HALF, bool REST>
struct Runs {
    static constexpr int C = HALF && REST ? 4 : 2;
    // first element of run i, or -1
    static __device__ __forceinline__ int32_t at(const Dims& d, uint32_t lane, int i) {
        int32_t e, end;
        if constexpr (HALF) {
            const int32_t own = (int32_t)lane * N;
            e = i == 0 ? own : i == 1 ? d.R / 2 + own : d.R + (int32_t)(lane + (i - 2) * d.lanes) * N;
            end = i == 0 ? d.R / 2 : i == 1 ? d.R : d.d;
        } else {
            e = (int32_t)(lane + i * d.lanes) * N, end = d.d;
        }
        return e < end ? e : -1;
    }
    float c[N], s[N];  // half: of run 0's pairs; interleaved: of run 0's, then run 1's
    // the table's runs of a position; sign -1 turns back
    template <bool F32T>
    __device__ __forceinline__ void load(const Dims& d, int64_t pos, uint32_t lane, float sign) {
        const int64_t row = pos * d.R;
        if constexpr (HALF) {
            const int32_t e = (int32_t)lane * N;
#pragma unroll
            for (int j = 0; j < N; ++j) c[j] = 1.0f, s[j] = 0.0f;  // (of a lane without such a run: its zeros stay zeros)
            if (e < d.R / 2) {
                table_run<F32T>(d.table, row + e, c);
                table_run<F32T>(d.table, row + d.R / 2 + e, s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t e = at(d, lane, i);
                float ci[N / 2], si[N / 2];
#pragma unroll
                for (int j = 0; j < N / 2; ++j) ci[j] = 1.0f, si[j] = 0.0f;
                if (e >= 0 && e < d.R) {
                    table_run<F32T>(d.table, row + e / 2, ci);
                    table_run<F32T>(d.table, row + d.R / 2 + e / 2, si);
                }
#pragma unroll
                for (int j = 0; j < N / 2; ++j) c[i * N / 2 + j] = ci[j], s[i * N / 2 + j] = si[j];
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] *= sign;
    }
    __device__ __forceinline__ void turn(const Dims& d, uint32_t lane, float (&v)[C][N]) const {
        if constexpr (HALF) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float a = v[0][j], b = v[1][j];
                v[0][j] = __builtin_fmaf(a, c[j], -(b * s[j]));
                v[1][j] = __builtin_fmaf(b, c[j], a * s[j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t e = at(d, lane, i);
                if (e < 0 || e >= d.R) continue;  // (a turn by 0 would make NaN of infinities)
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float a = v[i][2 * j], b = v[i][2 * j + 1], cj = c[i * N / 2 + j], sj = s[i * N / 2 + j];
                    v[i][2 * j] = __builtin_fmaf(a, cj, -(b * sj));
                    v[i][2 * j + 1] = __builtin_fmaf(b, cj, a * sj);
                }
            }
        }
    }
};

// Vector accesses, U heads of one row to a group of lanes: their loads are on the way together, and the row's part of
// the table and the gains are read once for them. The heads are `units` apart, so that a wave's loads cover
// neighbouring heads.
template <class E, bool F32T, bool HALF, bool REST, int U>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(Part q, Part k, Dims d, uint32_t q_blocks) {
    constexpr int N = E::N;
    typedef Runs<N, HALF, REST> R;
    constexpr int C = R::C;
    const bool keys = blockIdx.x >= q_blocks;
    const Part& p = keys ? k : q;
    const uint32_t id = ((blockIdx.x - (keys ? q_blocks : 0)) * kThreads + threadIdx.x) >> d.shift;
    const uint32_t t = quotient(id, p.per_row), u = id - t * p.units;
    if (t >= d.T) return;
    const uint32_t lane = threadIdx.x & (d.lanes - 1);
    const int64_t pos = d.positions[t];
    const typename E::T* x = static_cast<const typename E::T*>(p.x) + t * p.x_rs;
    typename E::T* out = static_cast<typename E::T*>(p.out) + t * p.out_rs;
    U32x4 raw[U][C];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const uint32_t h = u + j * p.units;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t e = R::at(d, lane, i);
            raw[j][i] = U32x4{0u, 0u, 0u, 0u};
            if (h < p.heads && e >= 0) raw[j][i] = load16(x + h * p.x_hs + e);
        }
    }
    const bool inside = pos >= 0 && pos < d.max_position;
    if (!inside && !d.pass) return;
    R run;
    float w[C][N];
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) w[i][n] = 1.0f;
    if (inside) {
        run.template load<F32T>(d, pos, lane, 1.0f);
        if (p.w) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int32_t e = R::at(d, lane, i);
                if (e >= 0) load_gains(p.w, p.w_type, e, w[i]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const uint32_t h = u + j * p.units;
        if (inside) {
            float v[C][N], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                E::unpack(raw[j][i], v[i]);
#pragma unroll
                for (int n = 0; n < N; ++n) sum = __builtin_fmaf(v[i][n], v[i][n], sum);
            }
            const float r = rsqrt_hw(__builtin_fmaf(over_lanes(sum, d.lanes), d.inv_d, d.eps));
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int n = 0; n < N; ++n) v[i][n] = v[i][n] * r * w[i][n];
            run.turn(d, lane, v);
#pragma unroll
            for (int i = 0; i < C; ++i) raw[j][i] = E::pack(v[i]);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t e = R::at(d, lane, i);
            if (h < p.heads && e >= 0) store16(out + h * p.out_hs + e, raw[j][i]);
        }
    }
}

// part: [blocks, d] sums of the gains' gradients, the queries' blocks first; nullptr: no gains at all.
template <class E, bool F32T, bool HALF, bool REST, int U>
__global__ __launch_bounds__(kThreads) void qk_norm_grad_kernel(Part q, Part k, Dims d, uint32_t q_blocks,
                                                                float* __restrict__ part) {
    constexpr int N = E::N;
    typedef Runs<N, HALF, REST> R;
    constexpr int C = R::C;
    __shared__ float sums[kThreads * N * C];  // [groups][d]
    const bool keys = blockIdx.x >= q_blocks;
    const Part& p = keys ? k : q;
    const uint32_t block = blockIdx.x - (keys ? q_blocks : 0), blocks = keys ? gridDim.x - q_blocks : q_blocks;
    const uint32_t groups = kThreads >> d.shift, group = threadIdx.x >> d.shift, lane = threadIdx.x & (d.lanes - 1);
    const uint32_t all = (uint32_t)d.T * p.units;
    float w[C][N], dw[C][N];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = R::at(d, lane, i);
#pragma unroll
        for (int n = 0; n < N; ++n) w[i][n] = 1.0f, dw[i][n] = 0.0f;
        if (p.w && e >= 0) load_gains(p.w, p.w_type, e, w[i]);
    }
    for (uint32_t id = block * groups + group; id < all; id += blocks * groups) {
        const uint32_t t = quotient(id, p.per_row), u = id - t * p.units;
        const int64_t pos = d.positions[t];
        const typename E::T* x = static_cast<const typename E::T*>(p.x) + t * p.x_rs;
        const typename E::T* gy = static_cast<const typename E::T*>(p.g) + t * p.g_rs;
        typename E::T* out = static_cast<typename E::T*>(p.out) + t * p.out_rs;
        U32x4 xr[U][C], gr[U][C];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t h = u + j * p.units;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int32_t e = R::at(d, lane, i);
                xr[j][i] = gr[j][i] = U32x4{0u, 0u, 0u, 0u};
                if (h < p.heads && e >= 0) {
                    xr[j][i] = load16(x + h * p.x_hs + e);
                    gr[j][i] = load16(gy + h * p.g_hs + e);
                }
            }
        }
        const bool inside = pos >= 0 && pos < d.max_position;
        if (!inside && !d.pass) continue;
        R run;
        if (inside) run.template load<F32T>(d, pos, lane, -1.0f);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t h = u + j * p.units;
            if (inside) {
                float v[C][N], g[C][N], sum = 0.0f, along = 0.0f;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    E::unpack(xr[j][i], v[i]);
                    E::unpack(gr[j][i], g[i]);
#pragma unroll
                    for (int n = 0; n < N; ++n) sum = __builtin_fmaf(v[i][n], v[i][n], sum);
                }
                run.turn(d, lane, g);
                // (heads that there are not have x 0, and eps may be 0: no NaN of theirs may reach dw)
                const float r = h < p.heads ? rsqrt_hw(__builtin_fmaf(over_lanes(sum, d.lanes), d.inv_d, d.eps)) : 0.0f;
#pragma unroll
                for (int i = 0; i < C; ++i)
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        v[i][n] *= r;
                        const float gv = g[i][n] * v[i][n];
                        dw[i][n] += gv;
                        along = __builtin_fmaf(gv, w[i][n], along);
                        g[i][n] *= w[i][n];
                    }
                along = over_lanes(along, d.lanes) * d.inv_d;
#pragma unroll
                for (int i = 0; i < C; ++i) {
#pragma unroll
                    for (int n = 0; n < N; ++n) g[i][n] = r * __builtin_fmaf(-v[i][n], along, g[i][n]);
                    gr[j][i] = E::pack(g[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int32_t e = R::at(d, lane, i);
                if (h < p.heads && e >= 0) store16(out + h * p.out_hs + e, gr[j][i]);
            }
        }
    }
    if (!p.w) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = R::at(d, lane, i);
        if (e < 0) continue;
#pragma unroll
        for (int n = 0; n < N; ++n) sums[group * d.d + e + n] = dw[i][n];
    }
    __syncthreads();
    for (int32_t e = threadIdx.x; e < d.d; e += kThreads) {
        float sum = 0.0f;
        for (uint32_t j = 0; j < groups; ++j) sum += sums[j * d.d + e];
        part[(int64_t)blockIdx.x * d.d + e] = sum;
    }
}

// Single elements, of heads that are not whole aligned units of 16 bytes: a wave a head, lane l elements l, l + 64 ...
// (a lane takes its elements' partners from memory again). grad: the gradient, as above.
template <bool F32T, bool HALF>
__device__ __forceinline__ float turned(const Dims& d, int64_t pos, int32_t e, float v, float partner, float sign) {
    if (e >= d.R) return v;
    const bool first = HALF ? e < d.R / 2 : e % 2 == 0;
    const int32_t j = HALF ? (first ? e : e - d.R / 2) : e / 2;
    const float c = table_at<F32T>(d.table, pos * d.R + j), s = table_at<F32T>(d.table, pos * d.R + d.R / 2 + j) * sign;
    return first ? __builtin_fmaf(v, c, -(partner * s)) : __builtin_fmaf(v, c, partner * s);
}
template <bool HALF>
__device__ __forceinline__ int32_t partner_of(const Dims& d, int32_t e) {
    return e >= d.R ? e : HALF ? (e < d.R / 2 ? e + d.R / 2 : e - d.R / 2) : e ^ 1;
}

template <class E, bool F32T, bool HALF, bool GRAD>
__global__ __launch_bounds__(kThreads) void qk_norm_single_kernel(Part q, Part k, Dims d, uint32_t q_blocks,
                                                                  float* __restrict__ part) {
    constexpr int C = kMaxHead / 64, kGroups = kThreads / 64;
    __shared__ float sums[kGroups][kMaxHead];
    const bool keys = blockIdx.x >= q_blocks;
    const Part& p = keys ? k : q;
    const uint32_t block = blockIdx.x - (keys ? q_blocks : 0), blocks = keys ? gridDim.x - q_blocks : q_blocks;
    const uint32_t group = threadIdx.x / 64, lane = threadIdx.x & 63u;
    const uint32_t all = (uint32_t)d.T * p.heads;
    float w[C], pw[C], dw[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = (int32_t)lane + 64 * i;
        w[i] = pw[i] = 1.0f, dw[i] = 0.0f;
        if (p.w && e < d.d) {
            float f[1];
            load_gains(p.w, p.w_type, e, f), w[i] = f[0];
            load_gains(p.w, p.w_type, partner_of<HALF>(d, e), f), pw[i] = f[0];
        }
    }
    for (uint32_t id = block * kGroups + group; id < all; id += blocks * kGroups) {
        const uint32_t t = quotient(id, p.per_row), h = id - t * p.units;
        const int64_t pos = d.positions[t];
        const typename E::T* x = static_cast<const typename E::T*>(p.x) + t * p.x_rs + h * p.x_hs;
        const typename E::T* src = GRAD ? static_cast<const typename E::T*>(p.g) + t * p.g_rs + h * p.g_hs : x;
        typename E::T* out = static_cast<typename E::T*>(p.out) + t * p.out_rs + h * p.out_hs;
        const bool inside = pos >= 0 && pos < d.max_position;
        if (!inside && !d.pass) continue;
        typename E::T as_is[C];
        float v[C], y[C], sum = 0.0f, along = 0.0f;
        float pv[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t e = (int32_t)lane + 64 * i;
            v[i] = pv[i] = y[i] = 0.0f;
            if (e >= d.d) continue;
            as_is[i] = src[e];
            y[i] = E::load(as_is[i]);
            pv[i] = E::load(src[partner_of<HALF>(d, e)]);
            v[i] = GRAD ? E::load(x[e]) : y[i];
            sum = __builtin_fmaf(v[i], v[i], sum);
        }
        const float r = rsqrt_hw(__builtin_fmaf(over_lanes(sum, 64), d.inv_d, d.eps));
        if (inside) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int32_t e = (int32_t)lane + 64 * i;
                if (e >= d.d) continue;
                if (!GRAD) {
                    y[i] = turned<F32T, HALF>(d, pos, e, v[i] * r * w[i], pv[i] * r * pw[i], 1.0f);
                } else {
                    y[i] = turned<F32T, HALF>(d, pos, e, y[i], pv[i], -1.0f);
                    v[i] *= r;
                    dw[i] += y[i] * v[i];
                    along = __builtin_fmaf(y[i] * v[i], w[i], along);
                }
            }
            if (GRAD) {
                along = over_lanes(along, 64) * d.inv_d;
#pragma unroll
                for (int i = 0; i < C; ++i) y[i] = r * __builtin_fmaf(-v[i], along, y[i] * w[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t e = (int32_t)lane + 64 * i;
            if (e < d.d) out[e] = inside ? E::store(y[i]) : as_is[i];
        }
    }
    if (!GRAD || !p.w) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = (int32_t)lane + 64 * i;
        if (e < d.d) sums[group][e] = dw[i];
    }
    __syncthreads();
    if ((int32_t)threadIdx.x < d.d)
        part[(int64_t)blockIdx.x * d.d + threadIdx.x] =
            (sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
}

// The gains' gradients from the workgroups' sums: a workgroup 16 elements of the queries' (blockIdx.y 0) or the
// keys' gains, 64 sums at a time.
constexpr int kJoinThreads = 1024;
struct Join {
    void* out;  // nullptr: no gains
    int32_t type;
    uint32_t first, count;  // workgroups
};
__global__ __launch_bounds__(kJoinThreads) void qk_norm_join_kernel(const float* __restrict__ part, int32_t d, Join q,
                                                                    Join k) {
    __shared__ float sums[kJoinThreads];
    const Join j = blockIdx.y ? k : q;
    if (!j.out) return;
    const int32_t e = blockIdx.x * 16 + (int32_t)(threadIdx.x & 15u);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (e < d) {
        const float* at = part + (int64_t)j.first * d + e;
        uint32_t b = threadIdx.x >> 4;
        for (; b + 192 < j.count; b += 256) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] += at[(int64_t)(b + 64 * i) * d];
        }
        for (; b < j.count; b += 64) sum[0] += at[(int64_t)b * d];
    }
    sums[threadIdx.x] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    for (int half = kJoinThreads / 2; half >= 16; half /= 2) {
        __syncthreads();
        if ((int)threadIdx.x < half) sums[threadIdx.x] += sums[threadIdx.x + half];
    }
    if (threadIdx.x >= 16 || e >= d) return;
    const float v = sums[threadIdx.x];
    if (j.type == NRC_DTYPE_F32)
        static_cast<float*>(j.out)[e] = v;
    else if (j.type == NRC_DTYPE_F16)
        static_cast<_Float16*>(j.out)[e] = (_Float16)v;
    else
        static_cast<uint16_t*>(j.out)[e] = (uint16_t)to_bf16(v);
}

// Lanes of a head for its runs of n elements (Runs), a power of two.
uint32_t lanes_of(const QkNormArgs& a, int32_t n) {
    const int32_t units = a.half ? a.rotary_dim / 2 / n : (a.head_dim / n + 1) / 2;
    const int32_t rest = a.half ? ((a.head_dim - a.rotary_dim) / n + 1) / 2 : 0;
    uint32_t lanes = 1;
    while ((int32_t)lanes < units || (int32_t)lanes < rest) lanes *= 2;
    return lanes;
}

// Whole units of 16 bytes in every tensor?
bool vec_of(const QkNormArgs& a, int32_t n) {
    int64_t odd = a.head_dim % n | a.rotary_dim % n | (a.half ? a.rotary_dim / 2 % n : 0);
    uintptr_t at = (uintptr_t)a.table;
    for (const QkPart* p : {&a.q, &a.k}) {
        if (!p->x || !p->heads) continue;
        at |= (uintptr_t)p->x | (uintptr_t)p->out | (uintptr_t)p->g | (uintptr_t)p->w;
        odd |= (p->x_rs | p->x_hs | p->out_rs | p->out_hs | p->g_rs | p->g_hs) % n;
    }
    return odd == 0 && (at & 15) == 0;
}

Part part_of(const QkPart& p, int32_t u) {
    const uint32_t units = (uint32_t)(p.heads + u - 1) / u;
    return Part{p.x, p.g, p.out, p.w, p.x_rs, p.x_hs, p.g_rs, p.g_hs, p.out_rs, p.out_hs, p.w_type, (uint32_t)p.heads, units,
                div_by(units ? units : 1u)};
}

// Workgroups of a kernel that walks over the groups of heads: to each part as many as those fill, 8 a CU in all at most.
struct Grid {
    uint32_t q, k;
};
Grid walking_grid(int64_t T, const Part& pq, const Part& pk, uint32_t groups, int32_t num_cus) {
    const int64_t most = 8 * (int64_t)num_cus;
    const int64_t q = (T * pq.units + groups - 1) / groups, k = (T * pk.units + groups - 1) / groups;
    if (q + k <= most) return Grid{(uint32_t)q, (uint32_t)k};
    int64_t ks = most * k / (q + k);
    if (k > 0 && ks < 1) ks = 1;
    if (q > 0 && ks > most - 1) ks = most - 1;
    return Grid{(uint32_t)(q < most - ks ? q : most - ks), (uint32_t)(k < ks ? k : ks)};
}

void join(const QkNormArgs& a, const Grid& g, hipStream_t stream) {
    if (a.q.dw || a.k.dw)
        hipLaunchKernelGGL(qk_norm_join_kernel, dim3((a.head_dim + 15) / 16, 2), dim3(kJoinThreads), 0, stream, a.part,
                           a.head_dim, Join{a.q.dw, a.q.w_type, 0, g.q}, Join{a.k.dw, a.k.w_type, g.q, g.k});
}

template <class E, bool F32T, bool HALF, bool REST, int U>
void launch_vec(const QkNormArgs& a, hipStream_t stream) {
    const uint32_t lanes = lanes_of(a, E::N), groups = kThreads / lanes;
    const Dims d{a.T, a.max_position, a.positions, a.table, a.head_dim, a.rotary_dim, lanes,
                 (uint32_t)__builtin_ctz(lanes), 1.0f / (float)a.head_dim, a.eps, a.pass};
    if (!a.grad) {
        const Part q = part_of(a.q, U), k = part_of(a.k, U);
        const uint32_t qb = (uint32_t)((a.T * q.units + groups - 1) / groups), kb = (uint32_t)((a.T * k.units + groups - 1) / groups);
        hipLaunchKernelGGL((qk_norm_kernel<E, F32T, HALF, REST, U>), dim3(qb + kb), dim3(kThreads), 0, stream, q, k, d, qb);
        return;
    }
    constexpr int UG = U > 2 ? 2 : U;
    const Part q = part_of(a.q, UG), k = part_of(a.k, UG);
    const Grid g = walking_grid(a.T, q, k, groups, a.num_cus);
    if (g.q + g.k > 0)
        hipLaunchKernelGGL((qk_norm_grad_kernel<E, F32T, HALF, REST, UG>), dim3(g.q + g.k), dim3(kThreads), 0, stream, q, k,
                           d, g.q, a.part);
    join(a, g, stream);
}

template <class E, bool F32T, bool HALF>
void launch(const QkNormArgs& a, hipStream_t stream) {
    if (!vec_of(a, E::N)) {
        const Dims d{a.T, a.max_position, a.positions, a.table, a.head_dim, a.rotary_dim, 64, 6, 1.0f / (float)a.head_dim,
                     a.eps, a.pass};
        const Part q = part_of(a.q, 1), k = part_of(a.k, 1);
        const Grid g = walking_grid(a.T, q, k, kThreads / 64, a.num_cus);
        auto kernel = a.grad ? qk_norm_single_kernel<E, F32T, HALF, true> : qk_norm_single_kernel<E, F32T, HALF, false>;
        if (g.q + g.k > 0) hipLaunchKernelGGL(kernel, dim3(g.q + g.k), dim3(kThreads), 0, stream, q, k, d, g.q, a.part);
        join(a, g, stream);
        return;
    }
    // Several heads to a group where that leaves every CU 8 waves (a step's 16 rows: one each).
    const int64_t lanes = (a.T * (a.q.heads + a.k.heads)) * lanes_of(a, E::N);
    const bool many = lanes / 4 >= (int64_t)a.num_cus * 512;
    auto go = [&](auto rest) {
        constexpr bool RE = decltype(rest)::value;
        many ? launch_vec<E, F32T, HALF, RE, 4>(a, stream) : launch_vec<E, F32T, HALF, RE, 1>(a, stream);
    };
    if constexpr (HALF)
        a.head_dim > a.rotary_dim ? go(std::true_type{}) : go(std::false_type{});
    else
        go(std::false_type{});
}

template <class E>
void launch_type(const QkNormArgs& a, hipStream_t stream) {
    if (a.table_f32)
        a.half ? launch<E, true, true>(a, stream) : launch<E, true, false>(a, stream);
    else
        a.half ? launch<E, false, true>(a, stream) : launch<E, false, false>(a, stream);
}

}  // namespace

int64_t qk_norm_grad_workspace(int32_t d, int32_t num_cus) { return (int64_t)8 * num_cus * d * 4; }

int launch_qk_norm(const QkNormArgs& a, hipStream_t stream) {
    if (a.dtype == NRC_DTYPE_BF16)
        launch_type<Bf16>(a, stream);
    else if (a.dtype == NRC_DTYPE_F16)
        launch_type<F16>(a, stream);
    else
        launch_type<F32>(a, stream);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
