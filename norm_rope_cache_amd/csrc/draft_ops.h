// Internal launch interface of the operators on a drafted token's way to the
// cache and over it (draft_api.cpp): norms with the rotation, cells of 4 bits,
// attention over them, attention with a window. Arguments reach these functions
// already validated.
#pragma once

#include "cache_ops.h"
#include "div.h"

namespace nrc {

// The queries or the keys: [T, heads, head_dim] views, strides in elements.
struct QkPart {
    const void* x;
    const void* g;  // gradient of the outputs, with QkNormArgs::grad
    void* out;      // outputs, or x's gradient
    const void* w;  // [head_dim] gains, or nullptr
    void* dw;       // their gradient (with grad and w), of w's type
    int64_t x_rs, x_hs, g_rs, g_hs, out_rs, out_hs;
    int32_t w_type;  // NRC_DTYPE_*
    int32_t heads;   // 0: there are none
};

struct QkNormArgs {
    QkPart q, k;
    int32_t dtype;  // NRC_DTYPE_*
    int64_t T;
    int32_t head_dim, rotary_dim;
    const int64_t* positions;
    const void* table;  // [max_position, rotary_dim]
    bool table_f32;
    int64_t max_position;
    bool half, grad;
    bool pass;  // rows without a row of the table are copied
    float eps;
    float* part;  // the workspace, with gains to differentiate
    int32_t num_cus;
};

// Bytes of QkNormArgs::part.
int64_t qk_norm_grad_workspace(int32_t head_dim, int32_t num_cus);

int launch_qk_norm(const QkNormArgs& a, hipStream_t stream);

// Paged caches of 4 bits, [layers, num_blocks, H, page] by strides in bytes.
struct Fp4Cache {
    uint8_t* cache;
    int64_t layer_stride, block_stride, head_stride;
    uint32_t num_blocks, block_size;
};

// K and V rows of L layers, [L, T, H, 64] by strides in elements, and their slots.
struct Fp4Rows {
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_ls, k_rs, k_hs, v_ls, v_rs, v_hs;
    const int64_t* slots;  // [L, T] by slots_ls
    int64_t slots_ls;
    int64_t T;
    int32_t H, L;
};

int64_t fp4_page(int64_t block_size);  // bytes of a page of a head

int launch_fp4_store(const Fp4Rows& r, const Fp4Cache& c, hipStream_t stream);
int launch_fp4_load(const Fp4Rows& r, const Fp4Cache& c, uint16_t* k, uint16_t* v, bool fill, hipStream_t stream);

// How a shape is worked on: the kernel (many rows: keys shared through LDS), 16-row query tiles of a wave (few rows),
// a workgroup's waves, workgroups along the rows, the shares that a block's tiles are dealt into at most and the tiles of one.
// Many rows: the workgroups of all sequences, heads and shares to a row block; by_lengths: that many at most, their
// shares of at least `share` tiles worked out from the lengths.
struct WindowPlan {
    bool many, by_lengths;
    int32_t q_tiles, waves, row_blocks, splits, share, groups;
};

WindowPlan plan_window_attention(int32_t B, int32_t H, int32_t G, int32_t max_nodes, int64_t max_ctx, int32_t window,
                                 int32_t sinks, int32_t num_cus);
int64_t window_attention_workspace(const WindowPlan& p, int64_t T, int64_t heads, int32_t B);

struct WindowArgs {
    PagedCache kv;  // fp4: pages of 4 bits, the strides in bytes (page_stride is not used)
    TreeQueries tq;
    int32_t window, sinks;  // window 2^31 - 1: none
    bool fp4;
    uint16_t* out;  // [T, H G, 64]
    float* lse;     // [T, H G]
    float* part;      // splits > 1: the partial sums' rows, [., 64] then [., 2]
    int32_t* shares;  // by_lengths: [B, 3], each sequence's first group, its shares and their tiles
    WindowPlan plan;
    Div by_group, by_heads, by_splits, by_blocks, by_block;  // tq.G, tq.H, plan.splits, plan.row_blocks, kv.block_size
    uint32_t fill;                                 // NRC_ATTENTION_FILL_*
};

int launch_window_attention(const WindowArgs& a, hipStream_t stream);

}  // namespace nrc
