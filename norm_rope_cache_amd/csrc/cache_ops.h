// Internal launch interface of the operators around the cache (cache_api.cpp):
// rotary positions, attention over the paged cache, received attention
// weight, eviction. Arguments reach these functions already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nrc {

constexpr int kMaxRotaryPairs = 128;

// Pair j's angle per position (radians) and the cos and sin of that step.
struct RopeSteps {
    double angle[kMaxRotaryPairs], cos[kMaxRotaryPairs], sin[kMaxRotaryPairs];
};

struct RopeTableArgs {
    int64_t start, count;
    int32_t pairs;       // rotary_dim / 2
    int32_t half_width;  // width / 2 >= pairs: the pairs after them do not turn
    double magnitude;
    void* out;
    int32_t dtype;  // NRC_DTYPE_BF16 or NRC_DTYPE_F32
    int32_t num_cus;
};

int launch_rope_table(const RopeTableArgs& a, const RopeSteps& steps, hipStream_t stream);

struct RopeRotateArgs {
    const void* x;
    int32_t dtype;  // NRC_DTYPE_*
    int64_t T;
    int32_t H, head_dim;
    int64_t x_rs, x_hs;  // row and head strides, elements
    const int64_t* positions;
    const void* table;  // [max_position, rotary_dim]
    bool table_f32;
    int64_t max_position;
    int32_t rotary_dim;
    bool half, inverse;
    bool pass;  // rows without a row of the table are copied
    void* out;
    int64_t out_rs, out_hs;
};

int launch_rope_rotate(const RopeRotateArgs& a, hipStream_t stream);

// One layer's paged cache, [num_blocks, H, block_size, 128] as a strided
// view (strides in elements), and the sequences' block tables: key i of
// sequence b is page i % block_size of block tables[b * table_stride +
// i / block_size]. Blocks outside [0, num_blocks), and keys past
// table_width blocks, do not exist.
struct PagedCache {
    uint16_t* cache;
    int64_t block_stride, page_stride, head_stride;
    const int32_t* tables;
    int64_t table_stride;
    uint32_t table_width;
    uint32_t num_blocks;
    uint32_t block_size;
    int32_t bs_shift;  // log2(block_size), or -1 when not a power of two
};

// The queries: sequence b's nodes are rows q_starts[b] .. q_starts[b + 1] - 1
// of q [T, H G, 64], node i's own key is key ctx_lens[b] + i.
struct TreeQueries {
    const uint16_t* q;
    int64_t q_rs, q_hs;
    int32_t T, H, G, B;
    const int32_t* ctx_lens;
    const int32_t* q_starts;
    int32_t max_nodes, max_ctx;
    const uint32_t* mask;  // [T, mask_words] or nullptr (a chain: node i sees the nodes up to itself)
    int32_t mask_words;    // 32-bit words a row
    float scale, softcap;  // softcap 0: none
};

// How a shape is worked on: the kernel (many rows: keys shared through LDS),
// the 16-row query tiles a wave holds, a workgroup's waves, the workgroups along the
// rows. Few rows: the number of splits and the tiles of one. Many rows: splits 1
// (none) or 2 (by the lengths: into at most `groups` workgroups per row block, of
// at least split_tiles tiles each).
struct AttentionPlan {
    bool many;
    int32_t q_tiles, waves, row_blocks, splits, split_tiles, groups;
};

AttentionPlan plan_tree_attention(int32_t B, int32_t H, int32_t G, int32_t max_nodes, int64_t max_ctx, bool capped,
                                  int32_t num_cus);
// Bytes of TreeAttentionArgs::part and, behind it, shares.
int64_t tree_attention_workspace(const AttentionPlan& p, int64_t T, int64_t heads, int32_t B);

struct TreeAttentionArgs {
    PagedCache kv;
    TreeQueries tq;
    uint16_t* out;  // [T, H G, 64]
    float* lse;     // [T, H G]
    float* part;      // splits > 1: the partial sums' rows, [., 64] then [., 2]
    int32_t* shares;  // many rows: [B, 2], each sequence's first group and its splits
    AttentionPlan plan;
    uint32_t fill;  // NRC_ATTENTION_FILL_*
};

int launch_tree_attention(const TreeAttentionArgs& a, hipStream_t stream);

struct AttentionMassArgs {
    PagedCache kv;
    TreeQueries tq;
    const float* lse;      // [T, H G]
    const float* weights;  // [B, H, width] by strides, or nullptr (0)
    int64_t w_bs, w_hs;
    float decay;
    float* out;  // [B, H, width] by strides
    int64_t out_bs, out_hs;
    int64_t width;
    int32_t num_cus;
};

int launch_attention_mass(const AttentionMassArgs& a, hipStream_t stream);

struct KvEvictArgs {
    PagedCache kv;
    int32_t B, H;
    const int32_t* lens;
    const float* weights;  // [B, H, width] by strides
    int64_t w_bs, w_hs;
    const int32_t* positions;  // the same
    int64_t p_bs, p_hs;
    int64_t width;
    const int32_t* ends;
    int32_t sinks, recent, budget;
    float* new_weights;      // [B, H, budget]
    int32_t* new_positions;  // [B, H, budget]
    int32_t* new_lens;       // [B]
    int32_t* moves;          // the workspace
    int32_t max_moves;       // min(budget, width - budget), 0 when nothing can move
    int32_t blocks;          // kv_evict_blocks(budget)
};

// Bytes of KvEvictArgs::moves; workgroups along a list's places.
int64_t kv_evict_workspace(int64_t lists, int64_t width, int64_t max_moves, int64_t blocks);
int32_t kv_evict_blocks(int64_t budget);

int launch_kv_evict(const KvEvictArgs& a, hipStream_t stream);

}  // namespace nrc
