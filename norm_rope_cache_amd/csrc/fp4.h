// Cells of 4 bits: 64 elements of K and 64 of V in groups of 32, a group's codes in 16
// bytes (e2m1: sign, 0 .5 1 1.5 2 3 4 6; the even element in the low half of a byte)
// and its scale in one, 2^(byte - 127). A page of a head holds its block_size cells'
// K codes, V codes and scale dwords (K's two groups, then V's), each kind in one run.
#pragma once

#include "device_common.h"

namespace nrc {

constexpr int kFp4Codes = 32;                             // bytes of a cell's K (or V) codes
constexpr int kFp4Cell = 2 * kFp4Codes + 4;               // bytes of a cell
constexpr uint32_t kScaleLow = 7, kScaleHigh = 252;       // a stored scale's range: 2^-120 .. 2^125
constexpr uint32_t kScaleNan = 255;                       // of a cell that stands for NaN

// Bytes of a page of a head.
constexpr int64_t fp4_page_bytes(int64_t block_size) { return (block_size * kFp4Cell + 15) / 16 * 16; }

// The conversions take a scale's exponent bits alone (its sign and mantissa may hold anything), and 255 makes NaN.
template <int BYTE>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, BYTE));
}
// The 8 elements of a dword of codes as bf16.
__device__ __forceinline__ U32x4 fp4_open(uint32_t codes, float scale) {
    return U32x4{fp4_pair<0>(codes, scale), fp4_pair<1>(codes, scale), fp4_pair<2>(codes, scale), fp4_pair<3>(codes, scale)};
}
// 8 elements of bf16 as a dword of codes: nearest, ties to even, above 6 scale 6.
__device__ __forceinline__ uint32_t fp4_close(U32x4 v, float scale) {
    auto pair = [](uint32_t w) { return __builtin_bit_cast(nrc_bf16x2, w); };
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v.x), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v.y), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v.z), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, pair(v.w), scale, 3);
}

}  // namespace nrc
