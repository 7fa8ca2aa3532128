// The C entry points of the operators on a drafted token's way to the cache and
// over it (include/nrc.h): argument checks, then launches. Every check runs on
// the host before the first launch, so a non-zero status means nothing was
// enqueued.
#include <hip/hip_runtime.h>

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

// Are the rows of two views whose spans interleave (parts of one wider row) apart from each other?
bool rows_interleave(const Range& a, int64_t a_heads, int64_t a_hs, int64_t a_rs, const Range& b, int64_t b_heads,
                     int64_t b_hs, int64_t b_rs, int64_t d, int64_t eb) {
    if (a_rs != b_rs || a_rs == 0) return false;
    const int64_t row = a_rs * eb, in_a = ((a_heads - 1) * a_hs + d) * eb, in_b = ((b_heads - 1) * b_hs + d) * eb;
    const int64_t apart = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p) % row, behind = apart < 0 ? apart + row : apart;
    return behind >= in_a && in_b <= row - behind;
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
        if (!any_meet({w}, {r})) return false;
        return !rows_interleave(w, wh, whs, wrs, r, rh, rhs, rrs, head_dim, type_bytes(dtype));
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

}  // extern "C"
