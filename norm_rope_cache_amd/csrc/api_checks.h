// Argument checks that the C entry points of the operators around the cache share.
#pragma once

#include <math.h>

#include "../../include/nrc.h"
#include "cache_ops.h"
#include "status.h"

namespace nrc {

inline int64_t type_bytes(int32_t dtype) { return dtype == NRC_DTYPE_F32 ? 4 : 2; }

// Elements from the first to the last of a [T, H, d] view, plus one.
inline int64_t span(int64_t T, int64_t H, int64_t d, int64_t rs, int64_t hs) { return (T - 1) * rs + (H - 1) * hs + d; }

// Do elements [p, p + n) and [q, q + m), of 4 bytes unless said otherwise, meet?
inline bool meet(const void* p, int64_t n, const void* q, int64_t m, int p_bytes = 4, int q_bytes = 4) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return n > 0 && m > 0 && a < b + q_bytes * (uint64_t)m && b < a + p_bytes * (uint64_t)n;
}

constexpr int64_t kBig = (int64_t)1 << 40;

// A layer's cache view and block tables, checked (the pointers with need).
inline int32_t paged_cache(const char* what, const uint16_t* cache, int64_t num_blocks, int64_t block_size,
                    int64_t block_stride, int64_t page_stride, int64_t head_stride, int32_t H, const int32_t* tables,
                    int64_t table_stride, int64_t table_width, int32_t B, bool need, PagedCache* out) {
    if (H < 1) return fail(NRC_EINVAL, "%s: H = %d < 1", what, H);
    if (B < 0) return fail(NRC_EINVAL, "%s: B = %d < 0", what, B);
    if (H > 65535 || B > 65535) return fail(NRC_ENOTSUP, "%s: more than 65535 heads or sequences", what);
    if (num_blocks < 1 || block_size < 1) return fail(NRC_EINVAL, "%s: num_blocks and block_size must be >= 1", what);
    if (num_blocks > (((int64_t)1 << 31) - 1) / block_size)
        return fail(NRC_ENOTSUP, "%s: %lld x %lld slots do not fit 31 bits", what, (long long)num_blocks,
                    (long long)block_size);
    for (int64_t s : {block_stride, page_stride, head_stride}) {
        if (s < 0 || s > kBig) return fail(NRC_EINVAL, "%s: cache strides must lie in [0, 2^40]", what);
        if (s & 7) return fail(NRC_ENOTSUP, "%s: cache strides must be multiples of 8 elements (16-byte accesses)", what);
    }
    if (num_blocks * block_stride > (int64_t)1 << 60)
        return fail(NRC_EINVAL, "%s: cache strides too large", what);
    if (table_width < 1 || table_width > (((int64_t)1 << 31) - 1) / block_size || table_stride < 0 || table_stride > kBig)
        return fail(NRC_EINVAL, "%s: block tables of %lld blocks (at least 1, at most 2^31 keys), stride %lld", what,
                    (long long)table_width, (long long)table_stride);
    if (need && (!cache || !tables)) return fail(NRC_EINVAL, "%s: NULL cache or tables", what);
    if (!aligned(cache, 16) || !aligned(tables, 4))
        return fail(NRC_EINVAL, "%s: cache must be 16-byte, tables 4-byte aligned", what);
    int32_t shift = -1;
    if ((block_size & (block_size - 1)) == 0)
        for (shift = 0; ((int64_t)1 << shift) != block_size;) ++shift;
    *out = PagedCache{const_cast<uint16_t*>(cache), block_stride, page_stride, head_stride, tables, table_stride,
                           (uint32_t)table_width, (uint32_t)num_blocks, (uint32_t)block_size, shift};
    return NRC_OK;
}

// The sizes of the queries (no pointers).
inline int32_t query_sizes(const char* what, int32_t B, int64_t T, int32_t Hq, int32_t H, int32_t max_nodes, int64_t max_ctx) {
    if (B < 0 || T < 0 || H < 1 || Hq < 1)
        return fail(NRC_EINVAL, "%s: B >= 0, T >= 0, H >= 1 and Hq >= 1 must hold", what);
    if (Hq % H) return fail(NRC_ENOTSUP, "%s: %d query heads are not a multiple of %d KV heads", what, Hq, H);
    if (max_nodes < 1 || max_nodes > 65535)
        return fail(NRC_EINVAL, "%s: max_nodes = %d must lie in [1, 65535]", what, max_nodes);
    if (max_ctx < 0 || max_ctx > ((int64_t)1 << 31) - (1 << 17))
        return fail(NRC_EINVAL, "%s: max_ctx = %lld must lie in [0, 2^31 - 2^17]", what, (long long)max_ctx);
    // rows in 31 bits, a launch's threads in 32
    if (T > ((int64_t)1 << 30) || T * Hq > ((int64_t)1 << 31) - 1 || Hq > 65536 || B > 65535 || H > 65535 ||
        (int64_t)B * H * ((int64_t)max_nodes * (Hq / H) / 16 + 1) > ((int64_t)1 << 22))
        return fail(NRC_ENOTSUP, "%s: too many rows for one call", what);
    return NRC_OK;
}

inline int32_t queries(const char* what, const uint16_t* q, int64_t q_rs, int64_t q_hs, int64_t T, int32_t Hq, int32_t H,
                int32_t B, const int32_t* ctx_lens, const int32_t* q_starts, int32_t max_nodes, int64_t max_ctx,
                const int64_t* mask, int32_t mask_words, float scale, float softcap, TreeQueries* out) {
    if (int32_t rc = query_sizes(what, B, T, Hq, H, max_nodes, max_ctx)) return rc;
    if (q_rs < 0 || q_hs < 0 || q_rs > kBig || q_hs > kBig || (q_rs | q_hs) & 7)
        return fail(NRC_EINVAL, "%s: q strides must be multiples of 8 elements in [0, 2^40]", what);
    if ((mask == nullptr) != (mask_words == 0) || mask_words < 0)
        return fail(NRC_EINVAL, "%s: mask_words must be 0 exactly without a tree_mask", what);
    if (mask && ((int64_t)mask_words * 64 < max_nodes || mask_words > 1024))
        return fail(NRC_EINVAL, "%s: %d mask words do not hold %d nodes (or are more than 1024)", what, mask_words,
                    max_nodes);
    if (!(scale > 0.0f) || !isfinite(scale)) return fail(NRC_EINVAL, "%s: scale must be positive", what);
    if (!(softcap >= 0.0f) || !isfinite(softcap)) return fail(NRC_EINVAL, "%s: softcap must be 0 or positive", what);
    // (the factors worked out from them stay finite; a cap's scores are off by 2^-22 of it)
    if (scale < 0x1p-40f || scale > 0x1p40f) return fail(NRC_ENOTSUP, "%s: scale is outside [2^-40, 2^40]", what);
    if (softcap != 0.0f && (softcap < 0x1p-10f || softcap > 0x1p10f))
        return fail(NRC_ENOTSUP, "%s: softcap is neither 0 nor in [2^-10, 2^10]", what);
    if (B > 0 && T > 0 && (!q || !ctx_lens || !q_starts)) return fail(NRC_EINVAL, "%s: NULL q, ctx_lens or q_starts", what);
    if (!aligned(q, 16) || !aligned(ctx_lens, 4) || !aligned(q_starts, 4) || !aligned(mask, 8))
        return fail(NRC_EINVAL, "%s: q must be 16-byte, ctx_lens and q_starts 4-byte, tree_mask 8-byte aligned", what);
    *out = TreeQueries{q, q_rs, q_hs, (int32_t)T, H, Hq / H, B, ctx_lens, q_starts, max_nodes, (int32_t)max_ctx,
                            reinterpret_cast<const uint32_t*>(mask), 2 * mask_words, scale, softcap};
    return NRC_OK;
}

// Memory that a call reads or writes, in bytes.
struct Range {
    const void* p;
    int64_t bytes;
};
template <int W, int R>
bool any_meet(const Range (&written)[W], const Range (&read)[R]) {
    for (const Range& w : written)
        for (const Range& r : read)
            if (w.p && r.p && meet(w.p, w.bytes, r.p, r.bytes, 1, 1)) return true;
    return false;
}
// From the first of a layer's cells to the last (at most 2^62 bytes: strides go up to 2^40 elements).
inline Range cells_range(const PagedCache& c, int32_t H) {
    const __int128 elements = (__int128)(c.num_blocks - 1) * c.block_stride + (__int128)(c.block_size - 1) * c.page_stride +
                              (__int128)(H - 1) * c.head_stride + 2 * NRC_HEAD_DIM;
    return Range{c.cache, elements > ((int64_t)1 << 61) ? (int64_t)1 << 62 : 2 * (int64_t)elements};
}
inline Range tables_range(const PagedCache& c, int32_t B) {
    return Range{c.tables, 4 * ((B - 1) * c.table_stride + (int64_t)c.table_width)};
}

}  // namespace nrc
