// Element types of the operators on heads, and runs of a cos/sin table.
#pragma once

#include "device_common.h"

namespace nrc {

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

}  // namespace nrc
