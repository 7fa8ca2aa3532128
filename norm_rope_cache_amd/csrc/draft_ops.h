// Internal launch interface of the operators on a drafted token's way to the
// cache and over it (draft_api.cpp): norms with the rotation, cells of 4 bits,
// attention over them, attention with a window. Arguments reach these functions
// already validated.
#pragma once

#include "cache_ops.h"

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

}  // namespace nrc
