// The C entry points of the operators around the cache (include/nrc.h):
// argument checks, then launches. Every check runs on the host before the
// first launch, so a non-zero status means nothing was enqueued.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>

#include "../../include/nrc.h"
#include "cache_ops.h"
#include "status.h"

using nrc::aligned;
using nrc::fail;
using nrc::launch_status;
using nrc::num_cus;

namespace {

constexpr double kPi = 3.14159265358979323846;

// Each pair's angle per position (nrc.h, nrc_rope_table); a message, or NULL.
const char* rope_angles(int32_t R, double base, int32_t scaling, double factor, double original_max, double low,
                        double high, double* f) {
    const int32_t pairs = R / 2;
    if (!(base > 1.0) || !isfinite(base)) return "base must be above 1";
    if (scaling != NRC_ROPE_SCALE_NONE && (!(factor > 0.0) || !isfinite(factor))) return "factor must be positive";
    if (scaling == NRC_ROPE_SCALE_BASE && R <= 2) return "a scaled base needs more than one pair";
    if (scaling == NRC_ROPE_SCALE_BANDS || scaling == NRC_ROPE_SCALE_RAMP) {
        if (!(original_max > 0.0) || !isfinite(original_max)) return "original_max must be positive";
        if (!(low > 0.0) || !(high > low) || !isfinite(high)) return "0 < low < high must hold";
    }
    const double b = scaling == NRC_ROPE_SCALE_BASE ? base * pow(factor, (double)R / (R - 2)) : base;
    double lo = 0.0, hi = 0.0;
    if (scaling == NRC_ROPE_SCALE_RAMP) {
        const double per = R / (2.0 * log(base));
        lo = floor(per * log(original_max / (high * 2.0 * kPi)));
        hi = ceil(per * log(original_max / (low * 2.0 * kPi)));
        if (lo < 0.0) lo = 0.0;
        if (hi > pairs - 1.0) hi = pairs - 1.0;
    }
    for (int32_t j = 0; j < pairs; ++j) {
        double v = pow(b, -2.0 * j / R);
        double t = 0.0;
        switch (scaling) {
            case NRC_ROPE_SCALE_LINEAR:
                v /= factor;
                break;
            case NRC_ROPE_SCALE_BANDS:
                t = (original_max * v / (2.0 * kPi) - low) / (high - low);
                t = t < 0.0 ? 0.0 : t > 1.0 ? 1.0 : t;
                v *= (1.0 - t) / factor + t;
                break;
            case NRC_ROPE_SCALE_RAMP:
                t = (j - lo) / (hi - lo > 1e-3 ? hi - lo : 1e-3);
                t = t < 0.0 ? 0.0 : t > 1.0 ? 1.0 : t;
                v *= t / factor + (1.0 - t);
                break;
            default:
                break;
        }
        if (!isfinite(v * (double)NRC_ROPE_MAX_POSITION)) return "the scaling's angles are not finite";
        f[j] = v;
    }
    return nullptr;
}

int64_t type_bytes(int32_t dtype) { return dtype == NRC_DTYPE_F32 ? 4 : 2; }

// Elements from the first to the last of a [T, H, d] view, plus one.
int64_t span(int64_t T, int64_t H, int64_t d, int64_t rs, int64_t hs) { return (T - 1) * rs + (H - 1) * hs + d; }

// Do elements [p, p + n) and [q, q + m), of 4 bytes unless said otherwise, meet?
bool meet(const void* p, int64_t n, const void* q, int64_t m, int p_bytes = 4, int q_bytes = 4) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return n > 0 && m > 0 && a < b + q_bytes * (uint64_t)m && b < a + p_bytes * (uint64_t)n;
}

}  // namespace

extern "C" {

int32_t nrc_rope_table(int64_t start, int64_t count, int32_t rotary_dim, int32_t width, double base, int32_t scaling,
                       double factor, double original_max, double low, double high, double magnitude, void* out,
                       int32_t dtype, void* stream) {
    const char* what = "rope_table";
    if (dtype != NRC_DTYPE_BF16 && dtype != NRC_DTYPE_F32)
        return fail(NRC_ENOTSUP, "%s: table type %d (0 bf16, 2 FP32)", what, dtype);
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 2 * nrc::kMaxRotaryPairs)
        return fail(NRC_ENOTSUP, "%s: rotary_dim = %d is not even in [2, %d]", what, rotary_dim,
                    2 * nrc::kMaxRotaryPairs);
    if (width < rotary_dim || width % 2 || width > 4 * nrc::kMaxRotaryPairs)
        return fail(NRC_EINVAL, "%s: width = %d must be even, at least rotary_dim and at most %d", what, width,
                    4 * nrc::kMaxRotaryPairs);
    if (scaling < NRC_ROPE_SCALE_NONE || scaling > NRC_ROPE_SCALE_RAMP)
        return fail(NRC_EINVAL, "%s: scaling %d is unknown", what, scaling);
    if (!isfinite((float)magnitude)) return fail(NRC_EINVAL, "%s: magnitude is not finite in FP32", what);
    if (start < 0 || count < 0 || start > NRC_ROPE_MAX_POSITION || count > NRC_ROPE_MAX_POSITION - start)
        return fail(NRC_EINVAL, "%s: positions %lld .. + %lld must lie in [0, %lld)", what, (long long)start,
                    (long long)count, (long long)NRC_ROPE_MAX_POSITION);
    nrc::RopeSteps steps{};
    if (const char* m = rope_angles(rotary_dim, base, scaling, factor, original_max, low, high, steps.angle))
        return fail(NRC_EINVAL, "%s: %s", what, m);
    if (count == 0) return NRC_OK;
    if (!out) return fail(NRC_EINVAL, "%s: NULL out", what);
    if (!aligned(out, type_bytes(dtype))) return fail(NRC_EINVAL, "%s: out must be aligned to its elements", what);
    for (int32_t j = 0; j < rotary_dim / 2; ++j) {
        steps.cos[j] = cos(steps.angle[j]);
        steps.sin[j] = sin(steps.angle[j]);
    }
    nrc::RopeTableArgs a{start, count, rotary_dim / 2, width / 2, magnitude, out, dtype, num_cus()};
    return launch_status(nrc::launch_rope_table(a, steps, (hipStream_t)stream), what);
}

int32_t nrc_rope_rotate(const void* x, int32_t dtype, int64_t T, int32_t H, int32_t head_dim, int64_t x_row_stride,
                        int64_t x_head_stride, const int64_t* positions, const void* cos_sin, int32_t table_dtype,
                        int64_t max_position, int32_t rotary_dim, int32_t layout, int32_t inverse, void* out,
                        int64_t out_row_stride, int64_t out_head_stride, void* stream) {
    return nrc_rope_rotate_ex(x, dtype, T, H, head_dim, x_row_stride, x_head_stride, positions, cos_sin, table_dtype,
                              max_position, rotary_dim, layout, inverse, out, out_row_stride, out_head_stride, 0, stream);
}

int32_t nrc_rope_rotate_ex(const void* x, int32_t dtype, int64_t T, int32_t H, int32_t head_dim, int64_t x_row_stride,
                           int64_t x_head_stride, const int64_t* positions, const void* cos_sin, int32_t table_dtype,
                           int64_t max_position, int32_t rotary_dim, int32_t layout, int32_t inverse, void* out,
                           int64_t out_row_stride, int64_t out_head_stride, uint32_t flags, void* stream) {
    const char* what = "rope_rotate";
    if (flags & ~(uint32_t)NRC_ROPE_PASS_OUTSIDE) return fail(NRC_EINVAL, "%s: unknown flags 0x%x", what, flags);
    if (dtype < NRC_DTYPE_BF16 || dtype > NRC_DTYPE_F32)
        return fail(NRC_ENOTSUP, "%s: type %d (0 bf16, 1 FP16, 2 FP32)", what, dtype);
    if (table_dtype != NRC_DTYPE_BF16 && table_dtype != NRC_DTYPE_F32)
        return fail(NRC_ENOTSUP, "%s: table type %d (0 bf16, 2 FP32)", what, table_dtype);
    if (layout != NRC_ROPE_INTERLEAVED && layout != NRC_ROPE_HALF)
        return fail(NRC_EINVAL, "%s: layout %d (0 interleaved, 1 half)", what, layout);
    if (inverse != 0 && inverse != 1) return fail(NRC_EINVAL, "%s: inverse is 0 or 1", what);
    if (T < 0 || H < 1 || head_dim < 2) return fail(NRC_EINVAL, "%s: T >= 0, H >= 1 and head_dim >= 2 must hold", what);
    if (T > ((int64_t)1 << 23)) return fail(NRC_ENOTSUP, "%s: T = %lld rows are too many for one call", what, (long long)T);
    if ((int64_t)H * head_dim > 65536)
        return fail(NRC_ENOTSUP, "%s: %d heads of %d are more than 65536 elements", what, H, head_dim);
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim)
        return fail(NRC_EINVAL, "%s: rotary_dim = %d must be even in [2, head_dim]", what, rotary_dim);
    if (max_position < 1 || max_position > NRC_ROPE_MAX_POSITION)
        return fail(NRC_EINVAL, "%s: max_position must lie in [1, %lld]", what, (long long)NRC_ROPE_MAX_POSITION);
    if (T == 0) return NRC_OK;
    if (!x || !positions || !cos_sin || !out) return fail(NRC_EINVAL, "%s: NULL operand", what);
    const int64_t eb = type_bytes(dtype);
    if (!aligned(x, eb) || !aligned(out, eb) || !aligned(cos_sin, type_bytes(table_dtype)) || !aligned(positions, 8))
        return fail(NRC_EINVAL, "%s: operands must be aligned to their elements", what);
    const int64_t big = (int64_t)1 << 40;
    for (int64_t s : {x_row_stride, x_head_stride, out_row_stride, out_head_stride})
        if (s < 0 || s > big) return fail(NRC_EINVAL, "%s: strides must lie in [0, 2^40]", what);
    // written views: no two elements in one place
    const bool heads_in_rows = out_head_stride >= head_dim && (T == 1 || out_row_stride >= (H - 1) * out_head_stride + head_dim);
    const bool rows_in_heads = out_row_stride >= head_dim && (H == 1 || out_head_stride >= (T - 1) * out_row_stride + head_dim);
    if (!heads_in_rows && !rows_in_heads && !(H == 1 && (T == 1 || out_row_stride >= head_dim)))
        return fail(NRC_EINVAL, "%s: out's heads overlap", what);
    const bool in_place = x == out && x_row_stride == out_row_stride && x_head_stride == out_head_stride;
    if (!in_place) {
        if (meet(x, span(T, H, head_dim, x_row_stride, x_head_stride), out,
                 span(T, H, head_dim, out_row_stride, out_head_stride), (int)eb, (int)eb))
            return fail(NRC_EINVAL, "%s: out must be x itself or lie apart from it", what);
    }
    // other workgroups still read these
    const int64_t out_span = span(T, H, head_dim, out_row_stride, out_head_stride);
    if (meet(out, out_span, positions, T, (int)eb, 8) ||
        meet(out, out_span, cos_sin, max_position * rotary_dim, (int)eb, (int)type_bytes(table_dtype)))
        return fail(NRC_EINVAL, "%s: out must lie apart from positions and cos_sin", what);
    nrc::RopeRotateArgs a{x, dtype, T, H, head_dim, x_row_stride, x_head_stride, positions, cos_sin,
                          table_dtype == NRC_DTYPE_F32, max_position, rotary_dim, layout == NRC_ROPE_HALF, inverse != 0,
                          (flags & NRC_ROPE_PASS_OUTSIDE) != 0 && !in_place, out, out_row_stride, out_head_stride};
    return launch_status(nrc::launch_rope_rotate(a, (hipStream_t)stream), what);
}

}  // extern "C"

namespace {

constexpr int64_t kBig = (int64_t)1 << 40;

// A layer's cache view and block tables, checked (the pointers with need).
int32_t paged_cache(const char* what, const uint16_t* cache, int64_t num_blocks, int64_t block_size,
                    int64_t block_stride, int64_t page_stride, int64_t head_stride, int32_t H, const int32_t* tables,
                    int64_t table_stride, int64_t table_width, int32_t B, bool need, nrc::PagedCache* out) {
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
    *out = nrc::PagedCache{const_cast<uint16_t*>(cache), block_stride, page_stride, head_stride, tables, table_stride,
                           (uint32_t)table_width, (uint32_t)num_blocks, (uint32_t)block_size, shift};
    return NRC_OK;
}

// The sizes of the queries (no pointers).
int32_t query_sizes(const char* what, int32_t B, int64_t T, int32_t Hq, int32_t H, int32_t max_nodes, int64_t max_ctx) {
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

int32_t queries(const char* what, const uint16_t* q, int64_t q_rs, int64_t q_hs, int64_t T, int32_t Hq, int32_t H,
                int32_t B, const int32_t* ctx_lens, const int32_t* q_starts, int32_t max_nodes, int64_t max_ctx,
                const int64_t* mask, int32_t mask_words, float scale, float softcap, nrc::TreeQueries* out) {
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
    *out = nrc::TreeQueries{q, q_rs, q_hs, (int32_t)T, H, Hq / H, B, ctx_lens, q_starts, max_nodes, (int32_t)max_ctx,
                            reinterpret_cast<const uint32_t*>(mask), 2 * mask_words, scale, softcap};
    return NRC_OK;
}

// A [B, H, width] view of 4-byte elements.
int32_t per_cell(const char* what, const char* name, const void* p, int64_t bs, int64_t hs, bool need) {
    if (need && !p) return fail(NRC_EINVAL, "%s: NULL %s", what, name);
    if (!aligned(p, 4)) return fail(NRC_EINVAL, "%s: %s must be 4-byte aligned", what, name);
    if (bs < 0 || hs < 0 || bs > kBig || hs > kBig)
        return fail(NRC_EINVAL, "%s: strides of %s must lie in [0, 2^40]", what, name);
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
Range cells_range(const nrc::PagedCache& c, int32_t H) {
    const __int128 elements = (__int128)(c.num_blocks - 1) * c.block_stride + (__int128)(c.block_size - 1) * c.page_stride +
                              (__int128)(H - 1) * c.head_stride + 2 * NRC_HEAD_DIM;
    return Range{c.cache, elements > ((int64_t)1 << 61) ? (int64_t)1 << 62 : 2 * (int64_t)elements};
}
// Is every cell of a layer in memory of its own? So it is when each kind of step, from the smallest stride on, passes
// all that the smaller ones reach.
bool cells_apart(const nrc::PagedCache& c, int32_t H) {
    struct Step {
        int64_t stride, count;
    } steps[] = {{c.page_stride, (int64_t)c.block_size}, {c.head_stride, H}, {c.block_stride, (int64_t)c.num_blocks}};
    std::sort(steps, steps + 3, [](const Step& a, const Step& b) { return a.stride < b.stride; });
    __int128 reach = 2 * NRC_HEAD_DIM;
    for (const Step& s : steps) {
        if (s.count == 1) continue;
        if (s.stride < reach) return false;
        reach += (__int128)(s.count - 1) * s.stride;
    }
    return true;
}
Range tables_range(const nrc::PagedCache& c, int32_t B) {
    return Range{c.tables, 4 * ((B - 1) * c.table_stride + (int64_t)c.table_width)};
}

int32_t max_moves(int64_t width, int32_t budget) {
    const int64_t over = width - budget;
    return over <= 0 ? 0 : (int32_t)(over < budget ? over : budget);
}

}  // namespace

extern "C" {

int64_t nrc_context_tree_attention_workspace_bytes(int32_t B, int64_t T, int32_t Hq, int32_t H, int32_t max_nodes,
                                                   int64_t max_ctx) {
    if (int32_t rc = query_sizes("context_tree_attention", B, T, Hq, H, max_nodes, max_ctx)) return rc;
    if (B == 0 || T == 0) return 0;
    int64_t bytes[2];  // without and with a softcap
    for (int capped = 0; capped < 2; ++capped)
        bytes[capped] = nrc::tree_attention_workspace(
            nrc::plan_tree_attention(B, H, Hq / H, max_nodes, max_ctx, capped, num_cus()), T, Hq, B);
    return bytes[0] > bytes[1] ? bytes[0] : bytes[1];
}

int32_t nrc_context_tree_attention(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int64_t T,
                                   int32_t Hq, const uint16_t* cache, int64_t num_blocks, int64_t block_size,
                                   int64_t block_stride, int64_t page_stride, int64_t head_stride, int32_t H,
                                   const int32_t* tables, int64_t table_stride, int64_t table_width, int32_t B,
                                   const int32_t* ctx_lens, const int32_t* q_starts, int32_t max_nodes,
                                   int64_t max_ctx, const int64_t* tree_mask, int32_t mask_words, float scale,
                                   float softcap, uint16_t* out, float* lse, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    return nrc_context_tree_attention_ex(q, q_row_stride, q_head_stride, T, Hq, cache, num_blocks, block_size, block_stride,
                                         page_stride, head_stride, H, tables, table_stride, table_width, B, ctx_lens,
                                         q_starts, max_nodes, max_ctx, tree_mask, mask_words, scale, softcap, out, lse,
                                         workspace, workspace_bytes, 0, stream);
}

int32_t nrc_context_tree_attention_ex(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int64_t T,
                                      int32_t Hq, const uint16_t* cache, int64_t num_blocks, int64_t block_size,
                                      int64_t block_stride, int64_t page_stride, int64_t head_stride, int32_t H,
                                      const int32_t* tables, int64_t table_stride, int64_t table_width, int32_t B,
                                      const int32_t* ctx_lens, const int32_t* q_starts, int32_t max_nodes,
                                      int64_t max_ctx, const int64_t* tree_mask, int32_t mask_words, float scale,
                                      float softcap, uint16_t* out, float* lse, void* workspace,
                                      int64_t workspace_bytes, uint32_t flags, void* stream) {
    const char* what = "context_tree_attention";
    if (flags & ~(uint32_t)(NRC_ATTENTION_FILL_OUT | NRC_ATTENTION_FILL_LSE))
        return fail(NRC_EINVAL, "%s: unknown flags 0x%x", what, flags);
    const bool work = B > 0 && T > 0;
    nrc::TreeAttentionArgs a{};
    if (int32_t rc = paged_cache(what, cache, num_blocks, block_size, block_stride, page_stride, head_stride, H, tables,
                                 table_stride, table_width, B, work, &a.kv))
        return rc;
    if (int32_t rc = queries(what, q, q_row_stride, q_head_stride, T, Hq, H, B, ctx_lens, q_starts, max_nodes, max_ctx,
                             tree_mask, mask_words, scale, softcap, &a.tq))
        return rc;
    if (!work && (T == 0 || flags == 0)) return NRC_OK;
    if (!out || !lse) return fail(NRC_EINVAL, "%s: NULL out or lse", what);
    if (!aligned(out, 16) || !aligned(lse, 4)) return fail(NRC_EINVAL, "%s: out must be 16-byte, lse 4-byte aligned", what);
    const Range out_range{out, T * Hq * 128}, lse_range{lse, T * Hq * 4},
        q_range{q, 2 * span(T, Hq, 64, q_row_stride, q_head_stride)};
    if (any_meet({out_range, lse_range}, {q_range}) || any_meet({out_range}, {lse_range}))
        return fail(NRC_EINVAL, "%s: q, out and lse must lie apart from each other", what);
    a.fill = flags;
    a.out = out;
    a.lse = lse;
    if (!work) return launch_status(nrc::launch_tree_attention(a, (hipStream_t)stream), what);
    a.plan = nrc::plan_tree_attention(B, H, Hq / H, max_nodes, max_ctx, softcap > 0.0f, num_cus());
    const int64_t bytes = nrc::tree_attention_workspace(a.plan, T, Hq, B);
    if (bytes > 0 && (!workspace || workspace_bytes < bytes || !aligned(workspace, 16)))
        return fail(NRC_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes", what, (long long)bytes);
    // other workgroups still read these
    const Range ws_range{workspace, bytes};
    if (any_meet({out_range, lse_range, ws_range},
                 {cells_range(a.kv, H), tables_range(a.kv, B), {ctx_lens, 4 * (int64_t)B}, {q_starts, 4 * ((int64_t)B + 1)},
                  {tree_mask, 8 * T * mask_words}}) ||
        any_meet({ws_range}, {q_range, out_range, lse_range}))
        return fail(NRC_EINVAL, "%s: out, lse and the workspace must lie apart from each other and the inputs", what);
    a.part = static_cast<float*>(workspace);
    if (bytes > 0 && a.plan.many)  // the last [B, 2] of it
        a.shares = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + bytes) - 2 * (int64_t)B;
    return launch_status(nrc::launch_tree_attention(a, (hipStream_t)stream), what);
}

int32_t nrc_context_attention_mass(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int64_t T,
                                   int32_t Hq, const uint16_t* cache, int64_t num_blocks, int64_t block_size,
                                   int64_t block_stride, int64_t page_stride, int64_t head_stride, int32_t H,
                                   const int32_t* tables, int64_t table_stride, int64_t table_width, int32_t B,
                                   const int32_t* ctx_lens, const int32_t* q_starts, int32_t max_nodes,
                                   int64_t max_ctx, const int64_t* tree_mask, int32_t mask_words, float scale,
                                   float softcap, const float* lse, const float* weights, int64_t w_batch_stride,
                                   int64_t w_head_stride, float decay, float* out, int64_t out_batch_stride,
                                   int64_t out_head_stride, int64_t width, void* stream) {
    const char* what = "context_attention_mass";
    if (width < 0 || width > ((int64_t)1 << 31) - (1 << 17))
        return fail(NRC_EINVAL, "%s: width = %lld must lie in [0, 2^31 - 2^17]", what, (long long)width);
    const bool work = B > 0 && width > 0;
    nrc::AttentionMassArgs a{};
    if (int32_t rc = paged_cache(what, cache, num_blocks, block_size, block_stride, page_stride, head_stride, H, tables,
                                 table_stride, table_width, B, work, &a.kv))
        return rc;
    if (int32_t rc = queries(what, q, q_row_stride, q_head_stride, T, Hq, H, B, ctx_lens, q_starts, max_nodes, max_ctx,
                             tree_mask, mask_words, scale, softcap, &a.tq))
        return rc;
    if (int32_t rc = per_cell(what, "weights", weights, w_batch_stride, w_head_stride, false)) return rc;
    if (int32_t rc = per_cell(what, "out", out, out_batch_stride, out_head_stride, work)) return rc;
    if (!isfinite(decay)) return fail(NRC_EINVAL, "%s: decay is not finite", what);
    if (!work) return NRC_OK;
    if (!ctx_lens || !q_starts || (T > 0 && !lse)) return fail(NRC_EINVAL, "%s: NULL ctx_lens, q_starts or lse", what);
    if (!aligned(lse, 4)) return fail(NRC_EINVAL, "%s: lse must be 4-byte aligned", what);
    const bool heads_in_rows = (H == 1 || out_head_stride >= width) &&
                               (B == 1 || out_batch_stride >= (H - 1) * out_head_stride + width);
    const bool rows_in_heads = (B == 1 || out_batch_stride >= width) &&
                               (H == 1 || out_head_stride >= (B - 1) * out_batch_stride + width);
    if (!heads_in_rows && !rows_in_heads) return fail(NRC_EINVAL, "%s: out's heads overlap", what);
    if (weights && weights == out && (w_batch_stride != out_batch_stride || w_head_stride != out_head_stride))
        return fail(NRC_EINVAL, "%s: weights that are out must have its strides", what);
    if (weights && weights != out && meet(weights, span(B, H, width, w_batch_stride, w_head_stride), out,
                                          span(B, H, width, out_batch_stride, out_head_stride)))
        return fail(NRC_EINVAL, "%s: weights must be out itself or lie apart from it", what);
    // other workgroups still read these
    if (any_meet({{out, 4 * span(B, H, width, out_batch_stride, out_head_stride)}},
                 {{q, T > 0 ? 2 * span(T, Hq, 64, q_row_stride, q_head_stride) : 0}, cells_range(a.kv, H), tables_range(a.kv, B),
                  {ctx_lens, 4 * (int64_t)B}, {q_starts, 4 * ((int64_t)B + 1)}, {tree_mask, 8 * T * mask_words},
                  {lse, 4 * T * Hq}}))
        return fail(NRC_EINVAL, "%s: out must lie apart from the inputs other than weights", what);
    a.lse = lse;
    a.weights = weights;
    a.w_bs = w_batch_stride;
    a.w_hs = w_head_stride;
    a.decay = decay;
    a.out = out;
    a.out_bs = out_batch_stride;
    a.out_hs = out_head_stride;
    a.width = width;
    a.num_cus = num_cus();
    return launch_status(nrc::launch_attention_mass(a, (hipStream_t)stream), what);
}

int64_t nrc_context_kv_evict_workspace_bytes(int32_t B, int32_t H, int64_t width, int32_t budget) {
    if (B < 0 || H < 1 || budget < 1 || width < 0 || width > ((int64_t)1 << 31) - (1 << 17))
        return fail(NRC_EINVAL, "context_kv_evict: B >= 0, H >= 1, budget >= 1 and 0 <= width < 2^31 - 2^17 must hold");
    return B == 0 ? 0 : nrc::kv_evict_workspace((int64_t)B * H, width, max_moves(width, budget),
                                                    nrc::kv_evict_blocks(budget));
}

int32_t nrc_context_kv_evict(uint16_t* cache, int64_t num_blocks, int64_t block_size, int64_t block_stride,
                             int64_t page_stride, int64_t head_stride, int32_t H, const int32_t* tables,
                             int64_t table_stride, int64_t table_width, int32_t B, const int32_t* lens,
                             const float* weights, int64_t w_batch_stride, int64_t w_head_stride,
                             const int32_t* positions, int64_t p_batch_stride, int64_t p_head_stride, int64_t width,
                             const int32_t* ends, int32_t sinks, int32_t recent, int32_t budget, float* new_weights,
                             int32_t* new_positions, int32_t* new_lens, void* workspace, int64_t workspace_bytes,
                             void* stream) {
    const char* what = "context_kv_evict";
    const int64_t bytes = nrc_context_kv_evict_workspace_bytes(B, H, width, budget);
    if (bytes < 0) return (int32_t)bytes;
    if (sinks < 0 || recent < 0) return fail(NRC_EINVAL, "%s: sinks and recent must be >= 0", what);
    const bool work = B > 0;
    nrc::KvEvictArgs a{};
    if (int32_t rc = paged_cache(what, cache, num_blocks, block_size, block_stride, page_stride, head_stride, H, tables,
                                 table_stride, table_width, B, work, &a.kv))
        return rc;
    if ((int64_t)B * H > 65535) return fail(NRC_ENOTSUP, "%s: more than 65535 heads of all sequences", what);
    if (work && !cells_apart(a.kv, H))
        return fail(NRC_EINVAL, "%s: cells of the cache overlap, and one's move would change another", what);
    const bool cells = work && width > 0;
    if (int32_t rc = per_cell(what, "weights", weights, w_batch_stride, w_head_stride, cells)) return rc;
    if (int32_t rc = per_cell(what, "positions", positions, p_batch_stride, p_head_stride, cells)) return rc;
    if (int32_t rc = per_cell(what, "new_weights", new_weights, 0, 0, work)) return rc;
    if (int32_t rc = per_cell(what, "new_positions", new_positions, 0, 0, work)) return rc;
    if (!work) return NRC_OK;
    if (!lens || !ends || !new_lens) return fail(NRC_EINVAL, "%s: NULL lens, ends or new_lens", what);
    if (!aligned(lens, 4) || !aligned(ends, 4) || !aligned(new_lens, 4))
        return fail(NRC_EINVAL, "%s: lens, ends and new_lens must be 4-byte aligned", what);
    if (bytes > 0 && (!workspace || workspace_bytes < bytes || !aligned(workspace, 16)))
        return fail(NRC_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes", what, (long long)bytes);
    // other workgroups still read these when one writes those
    const int64_t kept = 4 * (int64_t)B * H * budget;
    const Range nw{new_weights, kept}, np{new_positions, kept}, nl{new_lens, 4 * (int64_t)B}, ws{workspace, bytes},
        cells_moved = cells_range(a.kv, H);
    if (any_meet({nw, np, nl, ws, cells_moved},
                 {{weights, cells ? 4 * span(B, H, width, w_batch_stride, w_head_stride) : 0},
                  {positions, cells ? 4 * span(B, H, width, p_batch_stride, p_head_stride) : 0},
                  {lens, 4 * (int64_t)B},
                  {ends, 4 * (int64_t)B},
                  tables_range(a.kv, B)}) ||
        any_meet({nw, np, nl, ws}, {cells_moved}) || any_meet({nw}, {np, nl, ws}) || any_meet({np}, {nl, ws}) ||
        any_meet({nl}, {ws}))
        return fail(NRC_EINVAL,
                    "%s: new_weights, new_positions, new_lens, the workspace and the cache must lie apart from each "
                    "other and from the inputs",
                    what);
    a.B = B;
    a.H = H;
    a.lens = lens;
    a.weights = weights;
    a.w_bs = w_batch_stride;
    a.w_hs = w_head_stride;
    a.positions = positions;
    a.p_bs = p_batch_stride;
    a.p_hs = p_head_stride;
    a.width = width;
    a.ends = ends;
    a.sinks = sinks;
    a.recent = recent;
    a.budget = budget;
    a.new_weights = new_weights;
    a.new_positions = new_positions;
    a.new_lens = new_lens;
    a.moves = static_cast<int32_t*>(workspace);
    a.max_moves = max_moves(width, budget);
    a.blocks = nrc::kv_evict_blocks(budget);
    return launch_status(nrc::launch_kv_evict(a, (hipStream_t)stream), what);
}

}  // extern "C"
