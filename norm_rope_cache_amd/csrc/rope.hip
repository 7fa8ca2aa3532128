// Rotary positions: the cos/sin table and the rotation of heads by it.
//
// Pair j of a head with R rotary elements turns by p f_j at position p, f_j =
// base^(-2 j / R) with the scaling asked for (worked out on the host in
// double): (a, b) -> (a cos - b sin, b cos + a sin). The pairs are elements
// (2j, 2j + 1) ("interleaved", the page "...cutedsl.draft.context", _rope) or
// (j, j + R / 2) ("half"); elements from R on pass through.
//
// Table: an angle reaches 10^5 radians and more, where 24 bits leave nothing
// of the fraction of a turn, so angles are in double. A thread owns one pair
// of a run of positions: the run's first angle by a double sincos, the others
// by turning it by the pair's step (4 double operations, each step adding
// about 1e-16). Bound by the double sincos where there are few positions (a
// run of 1), by the double operations and 2-byte stores of a long table (131072
// positions of 64: 17 MB in 8.1 us).
//
// Rotation: reads x, writes as much, and 3 operations per element: bound by
// memory. One thread takes 16 bytes (interleaved: a run of whole pairs; half:
// 16 bytes of the first halves and the 16 that go with them) of one head of
// one row, so a wave covers whole heads with contiguous accesses. Products
// and sums in FP32, one rounding to the output type. 16384 rows of 64 heads of 64:
// 273 MB in 54.3 us (5.0 TB/s; a copy of 1 GiB reaches 5.1 to 5.2).
#include <type_traits>

#include "../../include/nrc.h"
#include "cache_ops.h"
#include "device_common.h"

namespace nrc {
namespace {

// k / d for k * d < 2^32 by one high product (d = 1: mul is 0).
struct SmallDiv {
    uint32_t mul, d;
};
SmallDiv small_div(uint32_t d) {
    return SmallDiv{d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d), d};
}
__device__ __forceinline__ uint32_t quotient(uint32_t k, SmallDiv s) { return s.mul ? __umulhi(k, s.mul) : k; }

template <bool F32>
__device__ __forceinline__ void put(void* out, int64_t i, float v) {
    if constexpr (F32)
        static_cast<float*>(out)[i] = v;
    else
        static_cast<uint16_t*>(out)[i] = (uint16_t)to_bf16(v);
}

// One thread: pair j (lanes along the pairs) of the positions run * RUN ...
template <bool F32>
__global__ __launch_bounds__(256) void rope_table_kernel(RopeSteps steps, int64_t start, int64_t count, int32_t pairs,
                                                         int32_t half_width, int32_t run, double magnitude,
                                                         void* __restrict__ out) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t r = id / half_width;
    const int32_t j = (int32_t)(id - r * half_width);
    const int64_t p0 = r * run;
    if (p0 >= count) return;
    const int64_t p1 = p0 + run < count ? p0 + run : count;
    const int64_t width = 2 * (int64_t)half_width;
    if (j >= pairs) {
        for (int64_t p = p0; p < p1; ++p) {
            put<F32>(out, p * width + j, 1.0f);
            put<F32>(out, p * width + half_width + j, 0.0f);
        }
        return;
    }
    double s, c;
    sincos((double)(start + p0) * steps.angle[j], &s, &c);
    const double dc = steps.cos[j], ds = steps.sin[j];
    for (int64_t p = p0; p < p1; ++p) {
        put<F32>(out, p * width + j, (float)(c * magnitude));
        put<F32>(out, p * width + half_width + j, (float)(s * magnitude));
        const double c2 = __builtin_fma(c, dc, -(s * ds));
        s = __builtin_fma(s, dc, c * ds);
        c = c2;
    }
}

// The element types: N elements in 16 bytes, to and from FP32.
struct Bf16 {
    typedef uint16_t T;
    static constexpr int N = 8;
    static __device__ __forceinline__ float load(T v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ T store(float v) { return (T)to_bf16(v); }
    static __device__ __forceinline__ void unpack(U32x4 w, float (&f)[8]) {
        f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
    }
    static __device__ __forceinline__ U32x4 pack(const float (&f)[8]) {
        // the paired conversion, unless there is a NaN (whose bits it does not keep to 0x7FC0)
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) nan |= __builtin_isnan(f[i]);
        if (!nan)
            return U32x4{pack_bf16_pair_hw(f[0], f[1]), pack_bf16_pair_hw(f[2], f[3]), pack_bf16_pair_hw(f[4], f[5]),
                         pack_bf16_pair_hw(f[6], f[7])};
        return U32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
    }
};
struct F16 {
    typedef _Float16 T;
    static constexpr int N = 8;
    typedef _Float16 V __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ float load(T v) { return (float)v; }
    static __device__ __forceinline__ T store(float v) { return (T)v; }
    static __device__ __forceinline__ void unpack(U32x4 w, float (&f)[8]) {
        const V v = __builtin_bit_cast(V, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
    }
    static __device__ __forceinline__ U32x4 pack(const float (&f)[8]) {
        V v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (_Float16)f[i];
        return __builtin_bit_cast(U32x4, v);
    }
};
struct F32 {
    typedef float T;
    static constexpr int N = 4;
    static __device__ __forceinline__ float load(T v) { return v; }
    static __device__ __forceinline__ T store(float v) { return v; }
    static __device__ __forceinline__ void unpack(U32x4 w, float (&f)[4]) {
        f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ U32x4 pack(const float (&f)[4]) {
        return U32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
};

template <bool F32T>
__device__ __forceinline__ float table_at(const void* t, int64_t i) {
    if constexpr (F32T)
        return static_cast<const float*>(t)[i];
    else
        return __uint_as_float((uint32_t) static_cast<const uint16_t*>(t)[i] << 16);
}

// N consecutive table entries, aligned to their size (N 2, 4 or 8).
template <bool F32T, int N>
__device__ __forceinline__ void table_run(const void* t, int64_t i, float (&f)[N]) {
    if constexpr (F32T) {
        typedef float V __attribute__((ext_vector_type(N < 4 ? N : 4)));
        const V* p = reinterpret_cast<const V*>(static_cast<const float*>(t) + i);
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = p[k / 4][k % 4];
    } else {
        typedef uint32_t V __attribute__((ext_vector_type(N / 2)));
        const V v = *reinterpret_cast<const V*>(static_cast<const uint16_t*>(t) + i);
        if constexpr (N == 2) {
            f[0] = bf16_lo(v[0]), f[1] = bf16_hi(v[0]);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) f[k] = k % 2 ? bf16_hi(v[k / 2]) : bf16_lo(v[k / 2]);
        }
    }
}

struct RotateDims {
    int64_t T, x_rs, x_hs, out_rs, out_hs, max_position;
    int32_t rotary_dim, rows_per_block;
    uint32_t units_per_row;
    SmallDiv per_row, per_head;
    float sign;  // of the sine: -1 for the inverse
    bool pass;   // rows without a table row are copied, not left as they are
};

// Blocks: x the groups of rows_per_block rows, y the parts of a group. One
// thread one unit of one head of one row. VEC: a unit is 16 bytes
// (HALF: twice 16, of the two halves; past the rotary elements 16); else one
// pair, or one element that passes through.
template <class E, bool F32T, bool HALF, bool VEC>
__global__ __launch_bounds__(256) void rope_rotate_kernel(const typename E::T* x, const int64_t* __restrict__ positions,
                                                          const void* __restrict__ table, typename E::T* out,
                                                          RotateDims d) {
    const uint32_t k = blockIdx.y * 256 + threadIdx.x;
    const uint32_t row = quotient(k, d.per_row);
    const int64_t t = (int64_t)blockIdx.x * d.rows_per_block + row;
    if (row >= (uint32_t)d.rows_per_block || t >= d.T) return;
    const uint32_t in_row = k - row * d.per_row.d;
    const uint32_t h = quotient(in_row, d.per_head);
    const uint32_t u = in_row - h * d.per_head.d;
    const int64_t pos = positions[t];
    const typename E::T* src = x + t * d.x_rs + (int64_t)h * d.x_hs;
    typename E::T* dst = out + t * d.out_rs + (int64_t)h * d.out_hs;
    const int32_t R = d.rotary_dim;
    if (pos < 0 || pos >= d.max_position) {
        if (!d.pass) return;
        // the elements of the unit, as they are (a turn by 0 would make NaN of infinities)
        if constexpr (VEC) {
            constexpr int N = E::N;
            const int32_t turning = HALF ? R / 2 / N : 0;
            const int32_t e = (int32_t)u < turning ? (int32_t)u * N : (HALF ? R : 0) + ((int32_t)u - turning) * N;
            store16(dst + e, load16(src + e));
            if ((int32_t)u < turning) store16(dst + R / 2 + e, load16(src + R / 2 + e));
        } else if ((int32_t)u < R / 2) {
            dst[2 * u] = src[2 * u];
            dst[2 * u + 1] = src[2 * u + 1];
        } else {
            dst[R / 2 + u] = src[R / 2 + u];
        }
        return;
    }
    const int64_t cs = pos * R;

    if constexpr (VEC && HALF) {
        constexpr int N = E::N;
        const int32_t turning = R / 2 / N;
        if ((int32_t)u < turning) {
            const int32_t e = (int32_t)u * N;
            float a[N], b[N], c[N], s[N], y[N], z[N];
            E::unpack(load16(src + e), a);
            E::unpack(load16(src + R / 2 + e), b);
            table_run<F32T, N>(table, cs + e, c);
            table_run<F32T, N>(table, cs + R / 2 + e, s);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float si = s[i] * d.sign;
                y[i] = __builtin_fmaf(a[i], c[i], -(b[i] * si));
                z[i] = __builtin_fmaf(b[i], c[i], a[i] * si);
            }
            store16(dst + e, E::pack(y));
            store16(dst + R / 2 + e, E::pack(z));
        } else {
            const int32_t e = R + ((int32_t)u - turning) * N;
            store16(dst + e, load16(src + e));
        }
    } else if constexpr (VEC) {
        constexpr int N = E::N;
        const int32_t e = (int32_t)u * N;
        const U32x4 w = load16(src + e);
        if (e < R) {
            float a[N], c[N / 2], s[N / 2], y[N];
            E::unpack(w, a);
            table_run<F32T, N / 2>(table, cs + e / 2, c);
            table_run<F32T, N / 2>(table, cs + R / 2 + e / 2, s);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float si = s[i] * d.sign;
                y[2 * i] = __builtin_fmaf(a[2 * i], c[i], -(a[2 * i + 1] * si));
                y[2 * i + 1] = __builtin_fmaf(a[2 * i + 1], c[i], a[2 * i] * si);
            }
            store16(dst + e, E::pack(y));
        } else {
            store16(dst + e, w);
        }
    } else {
        if ((int32_t)u < R / 2) {
            const int32_t j = (int32_t)u;
            const int32_t ia = HALF ? j : 2 * j, ib = HALF ? j + R / 2 : 2 * j + 1;
            const float a = E::load(src[ia]), b = E::load(src[ib]);
            const float c = table_at<F32T>(table, cs + j), s = table_at<F32T>(table, cs + R / 2 + j) * d.sign;
            dst[ia] = E::store(__builtin_fmaf(a, c, -(b * s)));
            dst[ib] = E::store(__builtin_fmaf(b, c, a * s));
        } else {
            const int32_t e = R / 2 + (int32_t)u;
            dst[e] = src[e];
        }
    }
}

template <class E, bool F32T, bool HALF, bool VEC>
void rotate(const RopeRotateArgs& a, hipStream_t stream) {
    RotateDims d{};
    const int32_t R = a.rotary_dim;
    const uint32_t per_head = VEC ? (HALF ? R / 2 / E::N + (a.head_dim - R) / E::N : a.head_dim / E::N)
                                  : (uint32_t)(a.head_dim - R / 2);
    d.units_per_row = per_head * (uint32_t)a.H;
    d.rows_per_block = d.units_per_row >= 256 ? 1 : (int32_t)(256 / d.units_per_row);
    d.per_row = small_div(d.units_per_row);
    d.per_head = small_div(per_head);
    d.T = a.T, d.x_rs = a.x_rs, d.x_hs = a.x_hs, d.out_rs = a.out_rs, d.out_hs = a.out_hs;
    d.max_position = a.max_position, d.rotary_dim = R;
    d.sign = a.inverse ? -1.0f : 1.0f;
    d.pass = a.pass;
    const dim3 grid((uint32_t)((a.T + d.rows_per_block - 1) / d.rows_per_block),
                    (d.rows_per_block * d.units_per_row + 255) / 256);
    hipLaunchKernelGGL((rope_rotate_kernel<E, F32T, HALF, VEC>), grid, dim3(256), 0, stream,
                       static_cast<const typename E::T*>(a.x), a.positions, a.table, static_cast<typename E::T*>(a.out),
                       d);
}

template <class E>
void rotate_type(const RopeRotateArgs& a, hipStream_t stream) {
    // 16-byte accesses: of every head's start, of whole units, and of the
    // table's runs (their offsets are multiples of the runs' size then)
    const uintptr_t at = (uintptr_t)a.x | (uintptr_t)a.out | (uintptr_t)a.table;
    const int64_t strides = a.x_rs | a.x_hs | a.out_rs | a.out_hs | a.head_dim | a.rotary_dim;
    const bool vec = (at & 15) == 0 && strides % E::N == 0 && (!a.half || (a.rotary_dim / 2) % E::N == 0);
    auto go = [&](auto f32t, auto half) {
        constexpr bool F = decltype(f32t)::value, HF = decltype(half)::value;
        vec ? rotate<E, F, HF, true>(a, stream) : rotate<E, F, HF, false>(a, stream);
    };
    auto layout = [&](auto f32t) { a.half ? go(f32t, std::true_type{}) : go(f32t, std::false_type{}); };
    a.table_f32 ? layout(std::true_type{}) : layout(std::false_type{});
}

}  // namespace

int launch_rope_table(const RopeTableArgs& a, const RopeSteps& steps, hipStream_t stream) {
    // Runs of up to 16 positions to a sincos, shorter while the threads would
    // not give every CU 8 waves.
    int32_t run = 16;
    while (run > 1 && a.count * a.half_width / run < (int64_t)a.num_cus * 512) run /= 2;
    const int64_t threads = (a.count + run - 1) / run * a.half_width;
    const dim3 grid((uint32_t)((threads + 255) / 256));
    auto kernel = a.dtype == NRC_DTYPE_F32 ? rope_table_kernel<true> : rope_table_kernel<false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, steps, a.start, a.count, a.pairs, a.half_width, run,
                       a.magnitude, a.out);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_rope_rotate(const RopeRotateArgs& a, hipStream_t stream) {
    if (a.dtype == NRC_DTYPE_BF16)
        rotate_type<Bf16>(a, stream);
    else if (a.dtype == NRC_DTYPE_F16)
        rotate_type<F16>(a, stream);
    else
        rotate_type<F32>(a, stream);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
