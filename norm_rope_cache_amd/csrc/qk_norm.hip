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
// Both read and write each tensor once and are bound by memory. A head belongs to a
// group of lanes, 16 bytes a lane (the power of two that holds it, up to the 64
// of a wave; a head's sums go over its lanes by lane exchanges). In the half layout a
// lane takes the 16 bytes that its own are paired with from memory again: they lie
// in the lines that its wave reads anyway, and an exchange of 8 floats would cost
// more than the L1's read. Heads that are not 16-byte aligned or not whole units take
// single elements.
// The gains' gradients: a lane keeps the sums of its own elements over all heads of its
// group, a workgroup adds its groups in LDS, and a second launch adds the workgroups' sums
// in one fixed order (no atomics: the same bits every time).
#include <type_traits>

#include "../../include/nrc.h"
#include "draft_ops.h"
#include "element.h"

namespace nrc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHead = 256;

// n / d for n < 2^31.
struct Div {
    uint32_t mul, shift;  // mul 0: d = 1
};
Div div_by(uint32_t d) {
    if (d == 1) return Div{0, 0};
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return Div{(uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), s - 1};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, Div d) { return d.mul ? __umulhi(n, d.mul) >> d.shift : n; }

struct Part {
    const void* x;
    const void* g;  // backward: y's gradient
    void* out;      // y, or x's gradient
    const void* w;
    int64_t x_rs, x_hs, g_rs, g_hs, out_rs, out_hs;
    int32_t w_type;
    uint32_t heads;  // of a row
    Div per_row;
};
struct Dims {
    int64_t T, max_position;
    const int64_t* positions;
    const void* table;
    int32_t d, R;
    uint32_t lanes, shift;  // of a head, and the log of it
    float eps;
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

template <class E, int N>
__device__ __forceinline__ void load_run(const typename E::T* p, float (&f)[N]) {
    if constexpr (N == 1)
        f[0] = E::load(*p);
    else
        E::unpack(load16(p), f);
}
template <class E, int N>
__device__ __forceinline__ void store_run(typename E::T* p, const float (&f)[N]) {
    if constexpr (N == 1)
        *p = E::store(f[0]);
    else
        store16(p, E::pack(f));
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

// How the run of N elements from e on turns: its partner's first element, and the table.
template <bool F32T, bool HALF, int N>
struct Turn {
    static constexpr bool kInside = !HALF && N > 1;  // pairs lie within the run
    bool turns;
    int32_t partner;
    float c[kInside ? N / 2 : N], s[kInside ? N / 2 : N];

    __device__ __forceinline__ Turn(const Dims& d, int32_t e) {
        turns = e < d.R;
        partner = kInside || !turns ? e : HALF ? (e < d.R / 2 ? e + d.R / 2 : e - d.R / 2) : e ^ 1;
    }
    // sign: -1 turns back
    __device__ __forceinline__ void load(const Dims& d, int64_t pos, int32_t e, float sign) {
        if (!turns) return;
        const int64_t row = pos * d.R;
        if constexpr (N == 1) {
            const int32_t j = HALF ? (e < d.R / 2 ? e : e - d.R / 2) : e / 2;
            c[0] = table_at<F32T>(d.table, row + j);
            s[0] = table_at<F32T>(d.table, row + d.R / 2 + j);
        } else {
            const int32_t j = HALF ? (e < d.R / 2 ? e : e - d.R / 2) : e / 2;
            table_run<F32T>(d.table, row + j, c);
            table_run<F32T>(d.table, row + d.R / 2 + j, s);
        }
        // (the pair's second element turns with +s times the first)
        const float f = kInside || (HALF ? e < d.R / 2 : e % 2 == 0) ? sign : -sign;
#pragma unroll
        for (float& v : s) v *= f;
    }
    // v turned; p: the partners.
    __device__ __forceinline__ void turn(float (&v)[N], const float (&p)[N]) const {
        if (!turns) return;
        if constexpr (kInside) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float a = v[2 * i], b = v[2 * i + 1];
                v[2 * i] = __builtin_fmaf(a, c[i], -(b * s[i]));
                v[2 * i + 1] = __builtin_fmaf(b, c[i], a * s[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __builtin_fmaf(v[i], c[i], -(p[i] * s[i]));
        }
    }
};

template <class E, bool F32T, bool HALF, bool VEC>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(Part q, Part k, Dims d, uint32_t q_blocks) {
    constexpr int N = VEC ? E::N : 1, C = VEC ? 1 : kMaxHead / 64;  // elements of a run, runs of a lane
    typedef Turn<F32T, HALF, N> T;
    const bool keys = blockIdx.x >= q_blocks;
    const Part p = keys ? k : q;
    const uint32_t id = ((blockIdx.x - (keys ? q_blocks : 0)) * kThreads + threadIdx.x) >> d.shift;
    const uint32_t t = quotient(id, p.per_row);
    if (t >= d.T) return;
    const uint32_t h = id - t * p.heads;
    const uint32_t lane = threadIdx.x & (d.lanes - 1);
    const int64_t pos = d.positions[t];
    const typename E::T* x = static_cast<const typename E::T*>(p.x) + t * p.x_rs + h * p.x_hs;
    typename E::T* out = static_cast<typename E::T*>(p.out) + t * p.out_rs + h * p.out_hs;
    const bool inside = pos >= 0 && pos < d.max_position;
    if (!inside && !d.pass) return;

    float v[C][N], pv[C][N], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = (int32_t)(lane + 64 * i) * N;
        if (e >= d.d) continue;
        const T turn(d, e);
        load_run<E>(x + e, v[i]);
        if (!T::kInside && turn.turns && inside) load_run<E>(x + turn.partner, pv[i]);
#pragma unroll
        for (int j = 0; j < N; ++j) sum = __builtin_fmaf(v[i][j], v[i][j], sum);
    }
    if (inside) {
        const float r = rsqrt_rn(over_lanes(sum, d.lanes) / (float)d.d + d.eps);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t e = (int32_t)(lane + 64 * i) * N;
            if (e >= d.d) continue;
            T turn(d, e);
            turn.load(d, pos, e, 1.0f);
            float w[N], pw[N];
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = pw[j] = 1.0f;
            if (p.w) {
                load_gains(p.w, p.w_type, e, w);
                if (!T::kInside && turn.turns) load_gains(p.w, p.w_type, turn.partner, pw);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                v[i][j] = v[i][j] * r * w[j];
                if (!T::kInside && turn.turns) pv[i][j] = pv[i][j] * r * pw[j];
            }
            turn.turn(v[i], pv[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = (int32_t)(lane + 64 * i) * N;
        if (e >= d.d) continue;
        if (inside)
            store_run<E>(out + e, v[i]);
        else if constexpr (VEC)  // (as it is, a NaN's bits too)
            store16(out + e, load16(x + e));
        else
            out[e] = x[e];
    }
}

// part: [blocks, d] sums of the gains' gradients, the queries' blocks first; nullptr: no gains at all.
template <class E, bool F32T, bool HALF, bool VEC>
__global__ __launch_bounds__(kThreads) void qk_norm_grad_kernel(Part q, Part k, Dims d, uint32_t q_blocks,
                                                                float* __restrict__ part) {
    constexpr int N = VEC ? E::N : 1, C = VEC ? 1 : kMaxHead / 64;
    typedef Turn<F32T, HALF, N> T;
    __shared__ float sums[kThreads * N * C];  // [groups][d]
    const bool keys = blockIdx.x >= q_blocks;
    const Part p = keys ? k : q;
    const uint32_t block = blockIdx.x - (keys ? q_blocks : 0), blocks = keys ? gridDim.x - q_blocks : q_blocks;
    const uint32_t groups = kThreads >> d.shift, group = threadIdx.x >> d.shift, lane = threadIdx.x & (d.lanes - 1);
    const uint32_t all = (uint32_t)d.T * p.heads;
    float w[C][N], dw[C][N];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = (int32_t)(lane + 64 * i) * N;
#pragma unroll
        for (int j = 0; j < N; ++j) w[i][j] = 1.0f, dw[i][j] = 0.0f;
        if (p.w && e < d.d) load_gains(p.w, p.w_type, e, w[i]);
    }
    const float inv_d = 1.0f / (float)d.d;
    for (uint32_t id = block * groups + group; id < all; id += blocks * groups) {
        const uint32_t t = quotient(id, p.per_row), h = id - t * p.heads;
        const int64_t pos = d.positions[t];
        const typename E::T* x = static_cast<const typename E::T*>(p.x) + t * p.x_rs + h * p.x_hs;
        const typename E::T* gy = static_cast<const typename E::T*>(p.g) + t * p.g_rs + h * p.g_hs;
        typename E::T* out = static_cast<typename E::T*>(p.out) + t * p.out_rs + h * p.out_hs;
        const bool inside = pos >= 0 && pos < d.max_position;
        if (!inside && !d.pass) continue;
        float v[C][N], g[C][N], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t e = (int32_t)(lane + 64 * i) * N;
            if (e >= d.d) continue;
            T turn(d, e);
            load_run<E>(x + e, v[i]);
            load_run<E>(gy + e, g[i]);
            if (inside) {
                float pg[N];
                if (!T::kInside && turn.turns) load_run<E>(gy + turn.partner, pg);
                turn.load(d, pos, e, -1.0f);
                turn.turn(g[i], pg);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) sum = __builtin_fmaf(v[i][j], v[i][j], sum);
        }
        if (inside) {
            const float r = rsqrt_rn(over_lanes(sum, d.lanes) / (float)d.d + d.eps);
            float along = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if ((int32_t)(lane + 64 * i) * N >= d.d) continue;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    v[i][j] *= r;
                    const float gv = g[i][j] * v[i][j];
                    dw[i][j] += gv;
                    along = __builtin_fmaf(gv, w[i][j], along);
                    g[i][j] *= w[i][j];
                }
            }
            along = over_lanes(along, d.lanes) * inv_d;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) g[i][j] = r * __builtin_fmaf(-v[i][j], along, g[i][j]);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int32_t e = (int32_t)(lane + 64 * i) * N;
            if (e >= d.d) continue;
            if (inside)
                store_run<E>(out + e, g[i]);
            else if constexpr (VEC)
                store16(out + e, load16(gy + e));
            else
                out[e] = gy[e];
        }
    }
    if (!p.w) return;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int32_t e = (int32_t)(lane + 64 * i) * N;
        if (e >= d.d) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) sums[group * d.d + e + j] = dw[i][j];
    }
    __syncthreads();
    for (int32_t e = threadIdx.x; e < d.d; e += kThreads) {
        float sum = 0.0f;
        for (uint32_t j = 0; j < groups; ++j) sum += sums[j * d.d + e];
        part[(int64_t)blockIdx.x * d.d + e] = sum;
    }
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

uint32_t lanes_of(int32_t d, int32_t n) {
    uint32_t lanes = 1;
    while (lanes < 64 && lanes * n < (uint32_t)d) lanes *= 2;
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

Part part_of(const QkPart& p) {
    return Part{p.x, p.g, p.out, p.w, p.x_rs, p.x_hs, p.g_rs, p.g_hs, p.out_rs, p.out_hs, p.w_type, (uint32_t)p.heads,
                div_by(p.heads ? (uint32_t)p.heads : 1u)};
}

// Workgroups of the gradient's kernel: to each part as many as its heads fill, 8 a CU in all at most.
struct GradGrid {
    uint32_t q, k;
};
GradGrid grad_grid(int64_t T, int64_t q_heads, int64_t k_heads, uint32_t groups, int32_t num_cus) {
    const int64_t most = 8 * (int64_t)num_cus;
    const int64_t q = (T * q_heads + groups - 1) / groups, k = (T * k_heads + groups - 1) / groups;
    if (q + k <= most) return GradGrid{(uint32_t)q, (uint32_t)k};
    int64_t ks = most * k / (q + k);
    if (k > 0 && ks < 1) ks = 1;
    if (q > 0 && ks > most - 1) ks = most - 1;
    return GradGrid{(uint32_t)(q < most - ks ? q : most - ks), (uint32_t)(k < ks ? k : ks)};
}

template <class E, bool F32T, bool HALF, bool VEC>
void launch(const QkNormArgs& a, hipStream_t stream) {
    constexpr int N = VEC ? E::N : 1;
    const uint32_t lanes = lanes_of(a.head_dim, N), groups = kThreads / lanes;
    const Dims d{a.T, a.max_position, a.positions, a.table, a.head_dim, a.rotary_dim, lanes,
                 (uint32_t)__builtin_ctz(lanes), a.eps, a.pass};
    const Part q = part_of(a.q), k = part_of(a.k);
    if (!a.grad) {
        const uint32_t qb = (uint32_t)((a.T * q.heads + groups - 1) / groups), kb = (uint32_t)((a.T * k.heads + groups - 1) / groups);
        hipLaunchKernelGGL((qk_norm_kernel<E, F32T, HALF, VEC>), dim3(qb + kb), dim3(kThreads), 0, stream, q, k, d, qb);
        return;
    }
    const GradGrid g = grad_grid(a.T, q.heads, k.heads, groups, a.num_cus);
    if (g.q + g.k > 0)
        hipLaunchKernelGGL((qk_norm_grad_kernel<E, F32T, HALF, VEC>), dim3(g.q + g.k), dim3(kThreads), 0, stream, q, k, d,
                           g.q, a.part);
    if (a.q.dw || a.k.dw)
        hipLaunchKernelGGL(qk_norm_join_kernel, dim3((a.head_dim + 15) / 16, 2), dim3(kJoinThreads), 0, stream, a.part,
                           a.head_dim, Join{a.q.dw, a.q.w_type, 0, g.q}, Join{a.k.dw, a.k.w_type, g.q, g.k});
}

template <class E>
void launch_type(const QkNormArgs& a, hipStream_t stream) {
    const bool vec = vec_of(a, E::N);
    auto go = [&](auto f32t, auto half) {
        constexpr bool F = decltype(f32t)::value, HF = decltype(half)::value;
        vec ? launch<E, F, HF, true>(a, stream) : launch<E, F, HF, false>(a, stream);
    };
    auto layout = [&](auto f32t) { a.half ? go(f32t, std::true_type{}) : go(f32t, std::false_type{}); };
    a.table_f32 ? layout(std::true_type{}) : layout(std::false_type{});
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
