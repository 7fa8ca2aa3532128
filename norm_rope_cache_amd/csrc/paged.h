// Device helpers of the kernels that read the paged cache.
#pragma once

#include "cache_ops.h"
#include "device_common.h"

namespace nrc {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma16(U32x4 a, U32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ __forceinline__ uint32_t block_of(uint32_t key, const PagedCache& c) {
    return c.bs_shift >= 0 ? key >> c.bs_shift : key / c.block_size;
}

// The key's entry of the table, an entry at all past its end.
__device__ __forceinline__ uint32_t page_of(const PagedCache& c, const int32_t* table, uint32_t key) {
    const uint32_t blk = block_of(key, c);
    return (uint32_t)table[blk < c.table_width ? blk : c.table_width - 1];
}
// Element offset of the key's 128-element run within head 0, by its entry, or -1
// where there is no such key.
__device__ __forceinline__ int64_t key_offset(const PagedCache& c, uint32_t key, uint32_t page) {
    const uint32_t blk = block_of(key, c);
    return blk < c.table_width && page < c.num_blocks
               ? (int64_t)page * c.block_stride + (int64_t)(key - blk * c.block_size) * c.page_stride
               : -1;
}
__device__ __forceinline__ int64_t key_offset(const PagedCache& c, const int32_t* table, uint32_t key) {
    const uint32_t blk = block_of(key, c);
    if (blk >= c.table_width) return -1;
    return key_offset(c, key, (uint32_t)table[blk]);
}

// A sequence's rows of q: the first, and how many (both within [0, T]).
struct Nodes {
    int32_t first, count;
};
__device__ __forceinline__ Nodes nodes_of(const TreeQueries& t, int32_t b) {
    const int32_t lo = t.q_starts[b], hi = t.q_starts[b + 1];
    Nodes n{lo, lo < 0 || hi > t.T || hi < lo ? 0 : hi - lo};
    if (n.count > t.max_nodes) n.count = t.max_nodes;
    return n;
}
__device__ __forceinline__ int32_t context_of(const TreeQueries& t, int32_t b) {
    const int32_t c = t.ctx_lens[b];
    return c < 0 ? 0 : c > t.max_ctx ? t.max_ctx : c;
}

// Bits 0 .. 31 of words[i]: does node `node` (< 0: no row) see keys key0 + 32 i .. of a sequence with ctx keys of
// context before its nodes.
template <int N>
__device__ __forceinline__ void seen_keys(uint32_t (&words)[N], const TreeQueries& t, const Nodes& nodes, int32_t ctx,
                                          int32_t node, int32_t key0) {
    const int32_t w0 = (key0 - ctx) >> 5;  // of the nodes' words of 32 (rounded down: the context's come before 0)
    uint32_t bits[N + 1];
#pragma unroll
    for (int i = 0; i <= N; ++i) bits[i] = 0xFFFFFFFFu;
    if (t.mask) {  // (every word on the way before the first is looked at)
        const uint32_t* row = t.mask + (int64_t)(nodes.first + (node < 0 ? 0 : node)) * t.mask_words;
#pragma unroll
        for (int i = 0; i <= N; ++i) {
            const int32_t w = w0 + i < t.mask_words ? w0 + i : t.mask_words - 1;
            bits[i] = row[w < 0 ? 0 : w];
        }
    }
    const int32_t last = t.mask ? nodes.count - 1 : node;  // the last node that can be seen
    auto word = [&](int i) {
        const int32_t behind = last - 32 * (w0 + i);  // how far it lies behind the word's first
        const uint32_t there = behind < 0 ? 0u : behind >= 31 ? 0xFFFFFFFFu : (2u << behind) - 1u;
        return node < 0 ? 0u : w0 + i < 0 ? 0xFFFFFFFFu : bits[i] & there;
    };
    uint32_t low = word(0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t high = word(i + 1);
        words[i] = __builtin_amdgcn_alignbit(high, low, (uint32_t)(key0 - ctx) & 31u);
        low = high;
    }
}

typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mfma32(U32x4 a, U32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
// S^T = K Q^T by v_mfma_f32_32x32x16_bf16: lane l holds, for row l % 32, the keys 8 (i / 4) + 4 (l / 32) + i % 4 of
// 32 at i = 0 .. 15. The bits of a word of 32 keys in that order:
__device__ __forceinline__ uint32_t bits_of_scores(uint32_t word, uint32_t half) {
    word >>= 4 * half;
    return (word & 0xFu) | (word >> 4 & 0xF0u) | (word >> 8 & 0xF00u) | (word >> 12 & 0xF000u);
}

// 16 bytes a lane from global memory to LDS at lds + 16 lane, without a register. As inline assembly, so
// that the kernel alone accounts for it (a wait for all of them before the barrier) instead of a wait before
// every LDS read (M0 is reserved: the compiler keeps nothing in it). An LDS DMA right after a write of M0 needs a wait state in between.
__device__ __forceinline__ void to_lds(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory");
}
// The same with 4 bytes a lane, at lds + 4 lane.
__device__ __forceinline__ void to_lds4(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(lds) : "memory");
}
// At most N of this wave's loads to LDS are still on the way (they land in order).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | (N >> 4) << 14 | 0x0F70);
    asm volatile("" ::: "memory");  // (LDS reads stay behind it)
}
// A barrier that waits for LDS accesses alone, not for loads on the way.
__device__ __forceinline__ void barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// This wave's loads to LDS have landed, and everybody's after the barrier.
__device__ __forceinline__ void landed() {
    wait_vmcnt<0>();
    __syncthreads();
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Sums over the lanes up to each one: within rows of 16 by shifts, then the
// rows' totals handed on (DPP: no LDS).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_0(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_inclusive(uint32_t v) {
    v += dpp_or_0<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v += dpp_or_0<0x112, 0xF>(v);
    v += dpp_or_0<0x114, 0xF>(v);
    v += dpp_or_0<0x118, 0xF>(v);
    v += dpp_or_0<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
    v += dpp_or_0<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
    return v;
}
__device__ __forceinline__ uint32_t wave_total(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)wave_inclusive(v), 63);
}
// The largest of the lanes', by the same steps.
__device__ __forceinline__ uint32_t wave_most(uint32_t v) {
    auto up = [&](uint32_t o) { v = v > o ? v : o; };
    up(dpp_or_0<0x111, 0xF>(v));
    up(dpp_or_0<0x112, 0xF>(v));
    up(dpp_or_0<0x114, 0xF>(v));
    up(dpp_or_0<0x118, 0xF>(v));
    up(dpp_or_0<0x142, 0xA>(v));
    up(dpp_or_0<0x143, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// e^x and log in base 2, the hardware's (relative error about 2^-23).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

}  // namespace nrc
