// The C entry points of the operators on a drafted token's way to the cache and
// over it (include/nrc.h): argument checks, then launches. Every check runs on
// the host before the first launch, so a non-zero status means nothing was
// enqueued.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <numeric>

#include "api_checks.h"
#include "draft_ops.h"

using namespace nrc;

namespace {

// One of the four tensors of the queries or the keys, [T, heads, d] by strides.
struct Rows3 {
    const char* name;
    const void* p;
    int64_t rs, hs;
    bool written;
};

bool type_known(int32_t t) { return t >= NRC_DTYPE_BF16 && t <= NRC_DTYPE_F32; }

// Do a [T, heads, d] view's elements lie in places of their own?
bool rows_apart(int64_t T, int64_t heads, int64_t d, int64_t rs, int64_t hs) {
    const bool heads_in_rows = (heads == 1 || hs >= d) && (T == 1 || rs >= (heads - 1) * hs + d);
    const bool rows_in_heads = (T == 1 || rs >= d) && (heads == 1 || hs >= (T - 1) * rs + d);
    return heads_in_rows || rows_in_heads;
}

// The sizes and the table that both directions share; `a` gets them.
int32_t qk_sizes(const char* what, int32_t dtype, int64_t T, int32_t head_dim, int32_t Hq, int32_t Hk, float eps,
                 const int64_t* positions, const void* cos_sin, int32_t table_dtype, int64_t max_position,
                 int32_t rotary_dim, int32_t layout, uint32_t flags, QkNormArgs* a) {
    if (flags & ~(uint32_t)NRC_ROPE_PASS_OUTSIDE) return fail(NRC_EINVAL, "%s: unknown flags 0x%x", what, flags);
    if (!type_known(dtype)) return fail(NRC_ENOTSUP, "%s: type %d (0 bf16, 1 FP16, 2 FP32)", what, dtype);
    if (table_dtype != NRC_DTYPE_BF16 && table_dtype != NRC_DTYPE_F32)
        return fail(NRC_ENOTSUP, "%s: table type %d (0 bf16, 2 FP32)", what, table_dtype);
    if (layout != NRC_ROPE_INTERLEAVED && layout != NRC_ROPE_HALF)
        return fail(NRC_EINVAL, "%s: layout %d (0 interleaved, 1 half)", what, layout);
    if (T < 0 || Hq < 1 || Hk < 0) return fail(NRC_EINVAL, "%s: T >= 0, Hq >= 1 and Hk >= 0 must hold", what);
    if (head_dim < 2 || head_dim > 256) return fail(NRC_ENOTSUP, "%s: head_dim = %d is not in [2, 256]", what, head_dim);
    if (T > ((int64_t)1 << 25) || T * ((int64_t)Hq + Hk) > ((int64_t)1 << 25))
        return fail(NRC_ENOTSUP, "%s: more than 2^25 heads in one call", what);
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim)
        return fail(NRC_EINVAL, "%s: rotary_dim = %d must be even in [2, head_dim]", what, rotary_dim);
    if (max_position < 1 || max_position > NRC_ROPE_MAX_POSITION)
        return fail(NRC_EINVAL, "%s: max_position must lie in [1, %lld]", what, (long long)NRC_ROPE_MAX_POSITION);
    if (!(eps >= 0.0f) || !isfinite(eps)) return fail(NRC_EINVAL, "%s: eps must be finite and at least 0", what);
    if (T > 0 && (!positions || !cos_sin)) return fail(NRC_EINVAL, "%s: NULL positions or cos_sin", what);
    if (!aligned(positions, 8) || !aligned(cos_sin, type_bytes(table_dtype)))
        return fail(NRC_EINVAL, "%s: positions and cos_sin must be aligned to their elements", what);
    a->dtype = dtype, a->T = T, a->head_dim = head_dim, a->rotary_dim = rotary_dim;
    a->positions = positions, a->table = cos_sin, a->table_f32 = table_dtype == NRC_DTYPE_F32;
    a->max_position = max_position, a->half = layout == NRC_ROPE_HALF, a->eps = eps;
    a->pass = (flags & NRC_ROPE_PASS_OUTSIDE) != 0, a->num_cus = num_cus();
    return NRC_OK;
}

template <int N>
int32_t qk_rows(const char* what, const QkNormArgs& a, int32_t heads, const Rows3 (&rows)[N]) {
    if (a.T == 0 || heads == 0) return NRC_OK;
    for (const Rows3& r : rows) {
        if (!r.p) return fail(NRC_EINVAL, "%s: NULL %s", what, r.name);
        if (!aligned(r.p, type_bytes(a.dtype))) return fail(NRC_EINVAL, "%s: %s must be aligned to its elements", what, r.name);
        if (r.rs < 0 || r.hs < 0 || r.rs > kBig || r.hs > kBig)
            return fail(NRC_EINVAL, "%s: strides of %s must lie in [0, 2^40]", what, r.name);
        if (r.written && !rows_apart(a.T, heads, a.head_dim, r.rs, r.hs))
            return fail(NRC_EINVAL, "%s: heads of %s overlap", what, r.name);
    }
    return NRC_OK;
}

int32_t gains(const char* what, const char* name, const void* w, int32_t type) {
    if (!w) return NRC_OK;
    if (!type_known(type)) return fail(NRC_ENOTSUP, "%s: type %d of %s (0 bf16, 1 FP16, 2 FP32)", what, type, name);
    if (!aligned(w, type_bytes(type))) return fail(NRC_EINVAL, "%s: %s must be aligned to its elements", what, name);
    return NRC_OK;
}

Range rows_range(const QkNormArgs& a, int32_t heads, const void* p, int64_t rs, int64_t hs) {
    return Range{a.T > 0 && heads > 0 ? p : nullptr, a.T > 0 && heads > 0 ? span(a.T, heads, a.head_dim, rs, hs) * type_bytes(a.dtype) : 0};
}

// A view's steps: their strides in elements and how many there are.
struct Step {
    int64_t stride, count;
};

// Are the elements of two views whose spans interleave apart from each other (parts of one wider row, heads of several
// tensors by turns)? `a` and `b` begin at multiples of eb bytes, their innermost runs are d elements. They are when, for
// some of the steps taken as a run of their own (what it spans), both runs lie apart in a period that all other steps of
// both are multiples of.
template <int N>
bool apart_by_steps(const void* a, const Step (&as)[N], const void* b, const Step (&bs)[N], int64_t d, int64_t eb) {
    const __int128 between = (__int128)(uintptr_t)b - (__int128)(uintptr_t)a;
    for (int inner = 0; inner < 1 << N; ++inner) {
        __int128 in_a = d, in_b = d;
        int64_t period = 0;
        for (int i = 0; i < N; ++i) {
            if (inner >> i & 1) {
                in_a += (__int128)(as[i].count - 1) * as[i].stride;
                in_b += (__int128)(bs[i].count - 1) * bs[i].stride;
            } else {
                if (as[i].count > 1) period = std::gcd(period, as[i].stride);
                if (bs[i].count > 1) period = std::gcd(period, bs[i].stride);
            }
        }
        if (period == 0) continue;  // (the spans themselves, which meet)
        __int128 behind = between % (period * (__int128)eb);
        if (behind < 0) behind += period * (__int128)eb;
        if (behind >= in_a * eb && in_b * eb <= period * (__int128)eb - behind) return true;
    }
    return false;
}

// A view of layers of 4-bit pages, checked (the pointer with need).
int32_t fp4_cache(const char* what, const uint8_t* caches, int64_t layer_stride, int64_t block_stride, int64_t head_stride,
                  int64_t num_blocks, int64_t block_size, int32_t H, bool need, Fp4Cache* out) {
    if (H < 1) return fail(NRC_EINVAL, "%s: H = %d < 1", what, H);
    if (num_blocks < 1 || block_size < 1) return fail(NRC_EINVAL, "%s: num_blocks and block_size must be >= 1", what);
    if (H > 65535) return fail(NRC_ENOTSUP, "%s: more than 65535 heads", what);
    if (num_blocks > (((int64_t)1 << 31) - 1) / block_size || block_size > ((int64_t)1 << 24))
        return fail(NRC_ENOTSUP, "%s: %lld x %lld slots do not fit 31 bits (a block 24)", what, (long long)num_blocks,
                    (long long)block_size);
    for (int64_t s : {layer_stride, block_stride, head_stride}) {
        if (s < 0 || s > kBig) return fail(NRC_EINVAL, "%s: cache strides must lie in [0, 2^40]", what);
        if (s & 15) return fail(NRC_ENOTSUP, "%s: cache strides must be multiples of 16 bytes", what);
    }
    if (num_blocks * block_stride > (int64_t)1 << 60) return fail(NRC_EINVAL, "%s: cache strides too large", what);
    if (need && !caches) return fail(NRC_EINVAL, "%s: NULL cache", what);
    if (!aligned(caches, 16)) return fail(NRC_EINVAL, "%s: the cache must be 16-byte aligned", what);
    *out = Fp4Cache{const_cast<uint8_t*>(caches), layer_stride, block_stride, head_stride, (uint32_t)num_blocks,
                    (uint32_t)block_size};
    return NRC_OK;
}
// From the first page's first byte to the last one's last.
Range pages_range(const Fp4Cache& c, int32_t H, int32_t L) {
    const __int128 bytes = (__int128)(L - 1) * c.layer_stride + (__int128)(c.num_blocks - 1) * c.block_stride +
                           (__int128)(H - 1) * c.head_stride + fp4_page(c.block_size);
    return Range{c.cache, bytes > ((int64_t)1 << 62) ? (int64_t)1 << 62 : (int64_t)bytes};
}
// Is every page in memory of its own?
bool pages_apart(const Fp4Cache& c, int32_t H, int32_t L) {
    Step steps[] = {{c.layer_stride, L}, {c.block_stride, (int64_t)c.num_blocks}, {c.head_stride, H}};
    std::sort(steps, steps + 3, [](const Step& a, const Step& b) { return a.stride < b.stride; });
    __int128 reach = fp4_page(c.block_size);
    for (const Step& s : steps) {
        if (s.count == 1) continue;
        if (s.stride < reach) return false;
        reach += (__int128)(s.count - 1) * s.stride;
    }
    return true;
}

// K's or V's rows, [L, T, H, 64] by strides in elements.
struct Rows4 {
    const char* name;
    const uint16_t* p;
    int64_t ls, rs, hs;
};
int32_t fp4_rows(const char* what, const Rows4& k, const Rows4& v, const int64_t* slots, int64_t slots_ls, int64_t T,
                 int32_t H, int32_t L, bool need, Fp4Rows* out) {
    if (T < 0 || L < 0) return fail(NRC_EINVAL, "%s: T >= 0 and L >= 0 must hold", what);
    if (T > ((int64_t)1 << 28) || T * H > ((int64_t)1 << 28) || L > 65535)
        return fail(NRC_ENOTSUP, "%s: too many rows or layers for one call", what);
    for (const Rows4* r : {&k, &v}) {
        if (need && !r->p) return fail(NRC_EINVAL, "%s: NULL %s", what, r->name);
        if (!aligned(r->p, 16)) return fail(NRC_EINVAL, "%s: %s must be 16-byte aligned", what, r->name);
        for (int64_t s : {r->ls, r->rs, r->hs})
            if (s < 0 || s > kBig || s & 7)
                return fail(NRC_EINVAL, "%s: strides of %s must be multiples of 8 elements in [0, 2^40]", what, r->name);
    }
    if (need && !slots) return fail(NRC_EINVAL, "%s: NULL slots", what);
    if (!aligned(slots, 8) || slots_ls < 0 || slots_ls > kBig)
        return fail(NRC_EINVAL, "%s: slots must be 8-byte aligned, their layer stride in [0, 2^40]", what);
    *out = Fp4Rows{k.p, v.p, k.ls, k.rs, k.hs, v.ls, v.rs, v.hs, slots, slots_ls, T, H, L};
    return NRC_OK;
}
Range rows4_range(const Rows4& r, int64_t T, int32_t H, int32_t L) {
    const __int128 n = (__int128)(L - 1) * r.ls + (__int128)(T - 1) * r.rs + (__int128)(H - 1) * r.hs + NRC_HEAD_DIM;
    return Range{r.p, n > ((int64_t)1 << 61) ? (int64_t)1 << 62 : 2 * (int64_t)n};
}
// Do rows that are written lie in places of their own (layers, rows and heads in any order)?
bool rows4_apart(const Rows4& r, int64_t T, int32_t H, int32_t L) {
    Step steps[] = {{r.ls, L}, {r.rs, T}, {r.hs, H}};
    std::sort(steps, steps + 3, [](const Step& a, const Step& b) { return a.stride < b.stride; });
    __int128 reach = NRC_HEAD_DIM;
    for (const Step& s : steps) {
        if (s.count == 1) continue;
        if (s.stride < reach) return false;
        reach += (__int128)(s.count - 1) * s.stride;
    }
    return true;
}

// The queries, outputs and workspace of both attentions; a->kv is set, cells what they read of the cache.
int32_t attend(const char* what, WindowArgs a, const Range& cells, const uint16_t* q, int64_t q_rs, int64_t q_hs, int64_t T,
               int32_t Hq, int32_t H, int32_t B, const int32_t* ctx_lens, const int32_t* q_starts, int32_t max_nodes,
               int64_t max_ctx, const int64_t* tree_mask, int32_t mask_words, float scale, float softcap, uint16_t* out,
               float* lse, void* workspace, int64_t workspace_bytes, uint32_t flags, void* stream) {
    if (flags & ~(uint32_t)(NRC_ATTENTION_FILL_OUT | NRC_ATTENTION_FILL_LSE))
        return fail(NRC_EINVAL, "%s: unknown flags 0x%x", what, flags);
    if (int32_t rc = queries(what, q, q_rs, q_hs, T, Hq, H, B, ctx_lens, q_starts, max_nodes, max_ctx, tree_mask, mask_words,
                             scale, softcap, &a.tq))
        return rc;
    const bool work = B > 0 && T > 0;
    if (!work && (T == 0 || flags == 0)) return NRC_OK;
    if (!out || !lse) return fail(NRC_EINVAL, "%s: NULL out or lse", what);
    if (!aligned(out, 16) || !aligned(lse, 4)) return fail(NRC_EINVAL, "%s: out must be 16-byte, lse 4-byte aligned", what);
    const Range out_range{out, T * Hq * 128}, lse_range{lse, T * Hq * 4}, q_range{q, 2 * span(T, Hq, 64, q_rs, q_hs)};
    if (any_meet({out_range, lse_range}, {q_range}) || any_meet({out_range}, {lse_range}))
        return fail(NRC_EINVAL, "%s: q, out and lse must lie apart from each other", what);
    a.fill = flags;
    a.out = out;
    a.lse = lse;
    if (!work) return launch_status(launch_window_attention(a, (hipStream_t)stream), what);
    a.plan = plan_window_attention(B, H, Hq / H, max_nodes, max_ctx, a.window, a.sinks, num_cus());
    const int64_t bytes = window_attention_workspace(a.plan, T, Hq, B);
    if (bytes > 0 && (!workspace || workspace_bytes < bytes || !aligned(workspace, 16)))
        return fail(NRC_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes", what, (long long)bytes);
    // other workgroups still read these
    const Range ws_range{workspace, bytes};
    if (any_meet({out_range, lse_range, ws_range},
                 {cells, tables_range(a.kv, B), {ctx_lens, 4 * (int64_t)B}, {q_starts, 4 * ((int64_t)B + 1)},
                  {tree_mask, 8 * T * mask_words}}) ||
        any_meet({ws_range}, {q_range, out_range, lse_range}))
        return fail(NRC_EINVAL, "%s: out, lse and the workspace must lie apart from each other and the inputs", what);
    a.part = static_cast<float*>(workspace);
    if (a.plan.by_lengths)  // the last [B, 3] of it
        a.shares = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + bytes) - 3 * (int64_t)B;
    return launch_status(launch_window_attention(a, (hipStream_t)stream), what);
}

int32_t window_sizes(const char* what, int32_t window, int32_t sinks) {
    if (window < 0 || sinks < 0) return fail(NRC_EINVAL, "%s: window and sinks must not be negative", what);
    return NRC_OK;
}

}  // namespace

extern "C" {

int32_t nrc_qk_norm_rotate(const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t Hq, const void* k,
                           int64_t k_row_stride, int64_t k_head_stride, int32_t Hk, int32_t dtype, int64_t T,
                           int32_t head_dim, const void* q_weight, int32_t q_weight_dtype, const void* k_weight,
                           int32_t k_weight_dtype, float eps, const int64_t* positions, const void* cos_sin,
                           int32_t table_dtype, int64_t max_position, int32_t rotary_dim, int32_t layout, void* out_q,
                           int64_t oq_row_stride, int64_t oq_head_stride, void* out_k, int64_t ok_row_stride,
                           int64_t ok_head_stride, uint32_t flags, void* stream) {
    const char* what = "qk_norm_rotate";
    QkNormArgs a{};
    if (int32_t rc = qk_sizes(what, dtype, T, head_dim, Hq, Hk, eps, positions, cos_sin, table_dtype, max_position,
                              rotary_dim, layout, flags, &a))
        return rc;
    if (int32_t rc = qk_rows(what, a, Hq, {{"q", q, q_row_stride, q_head_stride, false},
                                           {"out_q", out_q, oq_row_stride, oq_head_stride, true}}))
        return rc;
    if (int32_t rc = qk_rows(what, a, Hk, {{"k", k, k_row_stride, k_head_stride, false},
                                           {"out_k", out_k, ok_row_stride, ok_head_stride, true}}))
        return rc;
    if (int32_t rc = gains(what, "q_weight", q_weight, q_weight_dtype)) return rc;
    if (int32_t rc = gains(what, "k_weight", k_weight, k_weight_dtype)) return rc;
    if (T == 0) return NRC_OK;
    // in place (the same view), or apart; other workgroups still read the rest
    const bool q_in_place = q == out_q && q_row_stride == oq_row_stride && q_head_stride == oq_head_stride;
    const bool k_in_place = k == out_k && k_row_stride == ok_row_stride && k_head_stride == ok_head_stride;
    const Range rq = rows_range(a, Hq, q, q_row_stride, q_head_stride), rk = rows_range(a, Hk, k, k_row_stride, k_head_stride),
                ro = rows_range(a, Hq, out_q, oq_row_stride, oq_head_stride),
                rok = rows_range(a, Hk, out_k, ok_row_stride, ok_head_stride);
    if (any_meet({ro, rok}, {{positions, 8 * T},
                             {cos_sin, max_position * rotary_dim * type_bytes(table_dtype)},
                             {q_weight, head_dim * type_bytes(q_weight_dtype)},
                             {k_weight, head_dim * type_bytes(k_weight_dtype)}}))
        return fail(NRC_EINVAL, "%s: outputs must lie apart from positions, cos_sin and the gains", what);
    // (queries and keys of one projection's rows: their spans interleave, their heads do not meet)
    auto meets = [&](const Range& w, int64_t wrs, int64_t whs, int32_t wh, const Range& r, int64_t rrs, int64_t rhs, int32_t rh) {
        return any_meet({w}, {r}) && !apart_by_steps<2>(w.p, {{wrs, T}, {whs, wh}}, r.p, {{rrs, T}, {rhs, rh}}, head_dim,
                                                        type_bytes(dtype));
    };
    if ((!q_in_place && meets(ro, oq_row_stride, oq_head_stride, Hq, rq, q_row_stride, q_head_stride, Hq)) ||
        (!k_in_place && meets(rok, ok_row_stride, ok_head_stride, Hk, rk, k_row_stride, k_head_stride, Hk)) ||
        meets(ro, oq_row_stride, oq_head_stride, Hq, rk, k_row_stride, k_head_stride, Hk) ||
        meets(rok, ok_row_stride, ok_head_stride, Hk, rq, q_row_stride, q_head_stride, Hq) ||
        meets(ro, oq_row_stride, oq_head_stride, Hq, rok, ok_row_stride, ok_head_stride, Hk))
        return fail(NRC_EINVAL, "%s: an output must be its own input or lie apart from q, k and the other", what);
    a.q = QkPart{q, nullptr, out_q, q_weight, nullptr, q_row_stride, q_head_stride, 0, 0, oq_row_stride, oq_head_stride,
                 q_weight_dtype, Hq};
    a.k = QkPart{k, nullptr, out_k, k_weight, nullptr, k_row_stride, k_head_stride, 0, 0, ok_row_stride, ok_head_stride,
                 k_weight_dtype, Hk};
    return launch_status(launch_qk_norm(a, (hipStream_t)stream), what);
}

int64_t nrc_qk_norm_rotate_grad_workspace_bytes(int32_t head_dim, int32_t with_gains) {
    if (head_dim < 2 || head_dim > 256)
        return fail(NRC_ENOTSUP, "qk_norm_rotate_grad: head_dim = %d is not in [2, 256]", head_dim);
    return with_gains ? qk_norm_grad_workspace(head_dim, num_cus()) : 0;
}

int32_t nrc_qk_norm_rotate_grad(const void* grad_q, int64_t gq_row_stride, int64_t gq_head_stride, const void* grad_k,
                                int64_t gk_row_stride, int64_t gk_head_stride, const void* q, int64_t q_row_stride,
                                int64_t q_head_stride, int32_t Hq, const void* k, int64_t k_row_stride,
                                int64_t k_head_stride, int32_t Hk, int32_t dtype, int64_t T, int32_t head_dim,
                                const void* q_weight, int32_t q_weight_dtype, const void* k_weight,
                                int32_t k_weight_dtype, float eps, const int64_t* positions, const void* cos_sin,
                                int32_t table_dtype, int64_t max_position, int32_t rotary_dim, int32_t layout, void* dq,
                                void* dk, void* dq_weight, void* dk_weight, void* workspace, int64_t workspace_bytes,
                                uint32_t flags, void* stream) {
    const char* what = "qk_norm_rotate_grad";
    QkNormArgs a{};
    if (int32_t rc = qk_sizes(what, dtype, T, head_dim, Hq, Hk, eps, positions, cos_sin, table_dtype, max_position,
                              rotary_dim, layout, flags, &a))
        return rc;
    const int64_t dq_rs = (int64_t)Hq * head_dim, dk_rs = (int64_t)Hk * head_dim;
    if (int32_t rc = qk_rows(what, a, Hq, {{"q", q, q_row_stride, q_head_stride, false},
                                           {"grad_q", grad_q, gq_row_stride, gq_head_stride, false},
                                           {"dq", dq, dq_rs, head_dim, true}}))
        return rc;
    if (int32_t rc = qk_rows(what, a, Hk, {{"k", k, k_row_stride, k_head_stride, false},
                                           {"grad_k", grad_k, gk_row_stride, gk_head_stride, false},
                                           {"dk", dk, dk_rs, head_dim, true}}))
        return rc;
    if (int32_t rc = gains(what, "q_weight", q_weight, q_weight_dtype)) return rc;
    if (int32_t rc = gains(what, "k_weight", k_weight, k_weight_dtype)) return rc;
    const bool kw = k_weight && Hk > 0;
    if ((q_weight && !dq_weight) || (kw && !dk_weight)) return fail(NRC_EINVAL, "%s: NULL gradient of gains", what);
    if ((dq_weight && !q_weight) || (dk_weight && !kw)) return fail(NRC_EINVAL, "%s: a gradient of gains without gains", what);
    if (!aligned(dq_weight, type_bytes(q_weight_dtype)) || !aligned(dk_weight, type_bytes(k_weight_dtype)))
        return fail(NRC_EINVAL, "%s: gradients of gains must be aligned to their elements", what);
    const int64_t bytes = q_weight || kw ? qk_norm_grad_workspace(head_dim, a.num_cus) : 0;
    if (bytes > 0 && (!workspace || workspace_bytes < bytes || !aligned(workspace, 16)))
        return fail(NRC_EINVAL, "%s: needs a 16-byte aligned workspace of %lld bytes", what, (long long)bytes);
    if (T == 0 && bytes == 0) return NRC_OK;
    const Range written[] = {rows_range(a, Hq, dq, dq_rs, head_dim), rows_range(a, Hk, dk, dk_rs, head_dim),
                             {dq_weight, head_dim * type_bytes(q_weight_dtype)},
                             {dk_weight, head_dim * type_bytes(k_weight_dtype)},
                             {workspace, bytes}};
    if (any_meet(written, {rows_range(a, Hq, q, q_row_stride, q_head_stride), rows_range(a, Hk, k, k_row_stride, k_head_stride),
                           rows_range(a, Hq, grad_q, gq_row_stride, gq_head_stride),
                           rows_range(a, Hk, grad_k, gk_row_stride, gk_head_stride),
                           {positions, 8 * T},
                           {cos_sin, T > 0 ? max_position * rotary_dim * type_bytes(table_dtype) : 0},
                           {q_weight, head_dim * type_bytes(q_weight_dtype)},
                           {k_weight, head_dim * type_bytes(k_weight_dtype)}}))
        return fail(NRC_EINVAL, "%s: gradients and the workspace must lie apart from the inputs", what);
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (any_meet({written[i]}, {written[j]}))
                return fail(NRC_EINVAL, "%s: gradients and the workspace must lie apart from each other", what);
    a.grad = true;
    a.q = QkPart{q, grad_q, dq, q_weight, dq_weight, q_row_stride, q_head_stride, gq_row_stride, gq_head_stride, dq_rs,
                 head_dim, q_weight_dtype, Hq};
    a.k = QkPart{k, grad_k, dk, kw ? k_weight : nullptr, dk_weight, k_row_stride, k_head_stride, gk_row_stride,
                 gk_head_stride, dk_rs, head_dim, k_weight_dtype, Hk};
    a.part = static_cast<float*>(workspace);
    return launch_status(launch_qk_norm(a, (hipStream_t)stream), what);
}

int64_t nrc_fp4_page_bytes(int64_t block_size) {
    if (block_size < 1 || block_size > ((int64_t)1 << 24))
        return fail(NRC_EINVAL, "fp4_page_bytes: block_size = %lld must lie in [1, 2^24]", (long long)block_size);
    return fp4_page(block_size);
}

int32_t nrc_context_fp4_store(const uint16_t* k, int64_t k_layer_stride, int64_t k_row_stride, int64_t k_head_stride,
                              const uint16_t* v, int64_t v_layer_stride, int64_t v_row_stride, int64_t v_head_stride,
                              const int64_t* slots, int64_t slots_layer_stride, int64_t T, int32_t H, int32_t L,
                              uint8_t* caches, int64_t layer_stride, int64_t block_stride, int64_t head_stride,
                              int64_t num_blocks, int64_t block_size, void* stream) {
    const char* what = "context_fp4_store";
    const bool work = T > 0 && L > 0;
    Fp4Cache c{};
    Fp4Rows r{};
    const Rows4 kr{"k", k, k_layer_stride, k_row_stride, k_head_stride}, vr{"v", v, v_layer_stride, v_row_stride, v_head_stride};
    if (int32_t rc = fp4_cache(what, caches, layer_stride, block_stride, head_stride, num_blocks, block_size, H, work, &c))
        return rc;
    if (int32_t rc = fp4_rows(what, kr, vr, slots, slots_layer_stride, T, H, L, work, &r)) return rc;
    if (!work) return NRC_OK;
    if (!pages_apart(c, H, L)) return fail(NRC_EINVAL, "%s: pages of the caches overlap", what);
    if (any_meet({pages_range(c, H, L)}, {rows4_range(kr, T, H, L), rows4_range(vr, T, H, L),
                                          {slots, 8 * ((L - 1) * slots_layer_stride + T)}}))
        return fail(NRC_EINVAL, "%s: the caches must lie apart from k, v and slots", what);
    return launch_status(launch_fp4_store(r, c, (hipStream_t)stream), what);
}

int32_t nrc_context_fp4_load(const uint8_t* caches, int64_t layer_stride, int64_t block_stride, int64_t head_stride,
                             int64_t num_blocks, int64_t block_size, const int64_t* slots, int64_t slots_layer_stride,
                             int64_t T, int32_t H, int32_t L, uint16_t* k, int64_t k_layer_stride, int64_t k_row_stride,
                             int64_t k_head_stride, uint16_t* v, int64_t v_layer_stride, int64_t v_row_stride,
                             int64_t v_head_stride, uint32_t flags, void* stream) {
    const char* what = "context_fp4_load";
    if (flags & ~(uint32_t)NRC_FP4_FILL) return fail(NRC_EINVAL, "%s: unknown flags 0x%x", what, flags);
    const bool work = T > 0 && L > 0;
    Fp4Cache c{};
    Fp4Rows r{};
    const Rows4 kr{"k", k, k_layer_stride, k_row_stride, k_head_stride}, vr{"v", v, v_layer_stride, v_row_stride, v_head_stride};
    if (int32_t rc = fp4_cache(what, caches, layer_stride, block_stride, head_stride, num_blocks, block_size, H, work, &c))
        return rc;
    if (int32_t rc = fp4_rows(what, kr, vr, slots, slots_layer_stride, T, H, L, work, &r)) return rc;
    if (!work) return NRC_OK;
    if (!rows4_apart(kr, T, H, L) || !rows4_apart(vr, T, H, L)) return fail(NRC_EINVAL, "%s: rows of k or v overlap", what);
    const Range k_range = rows4_range(kr, T, H, L), v_range = rows4_range(vr, T, H, L);
    // (K and V side by side in a row, or head by head: their spans interleave, their rows do not meet)
    if (any_meet({k_range, v_range}, {pages_range(c, H, L), {slots, 8 * ((L - 1) * slots_layer_stride + T)}}) ||
        (any_meet({k_range}, {v_range}) && !apart_by_steps<3>(k, {{kr.ls, L}, {kr.rs, T}, {kr.hs, H}}, v,
                                                              {{vr.ls, L}, {vr.rs, T}, {vr.hs, H}}, NRC_HEAD_DIM, 2)))
        return fail(NRC_EINVAL, "%s: k and v must lie apart from each other, the caches and slots", what);
    return launch_status(launch_fp4_load(r, c, k, v, flags != 0, (hipStream_t)stream), what);
}

int64_t nrc_context_window_attention_workspace_bytes(int32_t B, int64_t T, int32_t Hq, int32_t H, int32_t max_nodes,
                                                     int64_t max_ctx, int32_t window, int32_t sinks) {
    const char* what = "context_window_attention";
    if (int32_t rc = query_sizes(what, B, T, Hq, H, max_nodes, max_ctx)) return rc;
    if (int32_t rc = window_sizes(what, window, sinks)) return rc;
    if (B == 0 || T == 0) return 0;
    return window_attention_workspace(plan_window_attention(B, H, Hq / H, max_nodes, max_ctx, window ? window : INT32_MAX,
                                                            window ? sinks : 0, num_cus()),
                                      T, Hq, B);
}

int32_t nrc_context_window_attention(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int64_t T, int32_t Hq,
                                     const uint16_t* cache, int64_t num_blocks, int64_t block_size, int64_t block_stride,
                                     int64_t page_stride, int64_t head_stride, int32_t H, const int32_t* tables,
                                     int64_t table_stride, int64_t table_width, int32_t B, const int32_t* ctx_lens,
                                     const int32_t* q_starts, int32_t max_nodes, int64_t max_ctx, const int64_t* tree_mask,
                                     int32_t mask_words, float scale, float softcap, int32_t window, int32_t sinks,
                                     uint16_t* out, float* lse, void* workspace, int64_t workspace_bytes, uint32_t flags,
                                     void* stream) {
    const char* what = "context_window_attention";
    WindowArgs a{};
    if (int32_t rc = paged_cache(what, cache, num_blocks, block_size, block_stride, page_stride, head_stride, H, tables,
                                 table_stride, table_width, B, B > 0 && T > 0, &a.kv))
        return rc;
    if (int32_t rc = window_sizes(what, window, sinks)) return rc;
    if (window < 1) return fail(NRC_EINVAL, "%s: window must be at least 1", what);
    a.window = window;
    a.sinks = sinks;
    return attend(what, a, cells_range(a.kv, H), q, q_row_stride, q_head_stride, T, Hq, H, B, ctx_lens, q_starts, max_nodes,
                  max_ctx, tree_mask, mask_words, scale, softcap, out, lse, workspace, workspace_bytes, flags, stream);
}

int32_t nrc_context_fp4_attention(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int64_t T, int32_t Hq,
                                  const uint8_t* cache, int64_t num_blocks, int64_t block_size, int64_t block_stride,
                                  int64_t head_stride, int32_t H, const int32_t* tables, int64_t table_stride,
                                  int64_t table_width, int32_t B, const int32_t* ctx_lens, const int32_t* q_starts,
                                  int32_t max_nodes, int64_t max_ctx, const int64_t* tree_mask, int32_t mask_words,
                                  float scale, float softcap, int32_t window, int32_t sinks, uint16_t* out, float* lse,
                                  void* workspace, int64_t workspace_bytes, uint32_t flags, void* stream) {
    const char* what = "context_fp4_attention";
    const bool work = B > 0 && T > 0;
    WindowArgs a{};
    Fp4Cache c{};
    if (int32_t rc = fp4_cache(what, cache, 0, block_stride, head_stride, num_blocks, block_size, H, work, &c)) return rc;
    // (the table's checks; the pages' are done)
    if (int32_t rc = paged_cache(what, reinterpret_cast<const uint16_t*>(cache), num_blocks, block_size, block_stride, 0,
                                 head_stride, H, tables, table_stride, table_width, B, work, &a.kv))
        return rc;
    if (int32_t rc = window_sizes(what, window, sinks)) return rc;
    a.fp4 = true;
    a.window = window ? window : INT32_MAX;
    a.sinks = window ? sinks : 0;
    return attend(what, a, pages_range(c, H, 1), q, q_row_stride, q_head_stride, T, Hq, H, B, ctx_lens, q_starts, max_nodes,
                  max_ctx, tree_mask, mask_words, scale, softcap, out, lse, workspace, workspace_bytes, flags, stream);
}

}  // extern "C"
