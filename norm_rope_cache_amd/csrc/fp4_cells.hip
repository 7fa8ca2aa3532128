// Rows of K and V into cells of 4 bits and back, all layers of a call in one
// launch.
//
// A group of 32 elements with the largest magnitude m gets the least power of
// two 2^e with m <= 6 2^e, so that no element saturates (e is held to -120 ..
// 125), and each element the nearest code of x / 2^e, ties to the even one. m's exponent
// and fraction say e: m = f 2^E with 1 <= f < 2 needs E - 2 up to f = 1.5, else E - 1.
// A cell with an infinity or NaN anywhere gets scale bytes of 255 and stands for NaN.
//
// Bound by memory: 256 bytes a cell on the bf16 side, 68 on the other. One
// lane takes one group: its 64 bytes in four loads that are on the way together,
// its maximum by packed 16-bit maxima of the magnitudes' bits, its codes by the
// hardware's conversion, two a time; the four lanes of a cell put its scale bytes
// together.
#include "../../include/nrc.h"
#include "draft_ops.h"
#include "fp4.h"

namespace nrc {
namespace {

constexpr int kThreads = 256;
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// The cell of a slot: its page's first byte in layer l's head h and its place there; false without one.
struct Cell {
    int64_t page;
    uint32_t at;
};
__device__ __forceinline__ bool cell_of(const Fp4Cache& c, int64_t slot, uint32_t l, uint32_t h, Cell* out) {
    if (slot < 0 || slot >= (int64_t)c.num_blocks * c.block_size) return false;
    const uint32_t block = c.bs_shift >= 0 ? (uint32_t)slot >> c.bs_shift : (uint32_t)slot / c.block_size;
    out->at = (uint32_t)slot - block * c.block_size;
    out->page = l * c.layer_stride + block * c.block_stride + h * c.head_stride;
    return true;
}
// Of the lane's group (0, 1 of K, 2, 3 of V): its codes' bytes in the page.
__device__ __forceinline__ int64_t codes_at(const Fp4Cache& c, const Cell& cell, uint32_t group) {
    return cell.page + (int64_t)(group >> 1) * kFp4Codes * c.block_size + cell.at * kFp4Codes + (group & 1u) * 16;
}
__device__ __forceinline__ int64_t scales_at(const Fp4Cache& c, const Cell& cell) {
    return cell.page + 2ll * kFp4Codes * c.block_size + cell.at * 4ll;
}

struct Unit {
    int64_t t;
    uint32_t h, l, group;
    bool there;
};
// Blocks: x the units of a layer, y the layers; 4 lanes a unit (row, head).
__device__ __forceinline__ Unit unit_of(const Fp4Rows& r) {
    const int64_t id = (int64_t)blockIdx.x * (kThreads / 4) + (threadIdx.x >> 2);
    Unit u;
    u.there = id < r.T * r.H;
    u.t = u.there ? (int64_t)((uint32_t)id / (uint32_t)r.H) : 0;
    u.h = u.there ? (uint32_t)id - (uint32_t)u.t * (uint32_t)r.H : 0u;
    u.l = blockIdx.y;
    u.group = threadIdx.x & 3u;
    return u;
}

__global__ __launch_bounds__(kThreads) void fp4_store_kernel(Fp4Rows r, Fp4Cache c) {
    const Unit u = unit_of(r);
    if (!u.there) return;  // (a unit's four lanes go together)
    Cell cell;
    if (!cell_of(c, r.slots[u.l * r.slots_ls + u.t], u.l, u.h, &cell)) return;
    const bool v = u.group >> 1;
    const uint16_t* src = v ? r.v + u.l * r.v_ls + u.t * r.v_rs + u.h * r.v_hs : r.k + u.l * r.k_ls + u.t * r.k_rs + u.h * r.k_hs;
    U32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = load16(src + 32 * (u.group & 1u) + 8 * i);
    u16x2 most{0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, (&x[i / 4].x)[i % 4] & 0x7FFF7FFFu));
    const uint32_t m = most.x > most.y ? most.x : most.y;
    // 1.5's fraction bits are 0x40; subnormals (exponent 0) end at the lowest scale
    uint32_t byte = m >> 7;
    const uint32_t down = (m & 0x7Fu) <= 0x40u ? 2u : 1u;
    byte = byte < kScaleLow + down ? kScaleLow : byte - down;
    byte = byte > kScaleHigh ? kScaleHigh : byte;
    const float scale = __uint_as_float(byte << 23);
    uint32_t bytes = byte << (8 * u.group), bad = m >= 0x7F80u;
    // the cell's four lanes (quad permutes)
    bytes |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bytes, 0xB1, 0xF, 0xF, true);
    bytes |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bytes, 0x4E, 0xF, 0xF, true);
    bad |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bad, 0xB1, 0xF, 0xF, true);
    bad |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bad, 0x4E, 0xF, 0xF, true);
    U32x4 codes{fp4_close(x[0], scale), fp4_close(x[1], scale), fp4_close(x[2], scale), fp4_close(x[3], scale)};
    if (bad) codes = U32x4{0u, 0u, 0u, 0u};
    store16(c.cache + codes_at(c, cell, u.group), codes);
    if (u.group == 0) *reinterpret_cast<uint32_t*>(c.cache + scales_at(c, cell)) = bad ? 0xFFFFFFFFu : bytes;
}

// fill: rows without a cell become 0, not left as they are.
__global__ __launch_bounds__(kThreads) void fp4_load_kernel(Fp4Rows r, Fp4Cache c, uint16_t* __restrict__ k,
                                                            uint16_t* __restrict__ v, bool fill) {
    const Unit u = unit_of(r);
    if (!u.there) return;
    Cell cell;
    const bool there = cell_of(c, r.slots[u.l * r.slots_ls + u.t], u.l, u.h, &cell);
    if (!there && !fill) return;
    U32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = U32x4{0u, 0u, 0u, 0u};
    if (there) {
        const U32x4 codes = load16(c.cache + codes_at(c, cell, u.group));
        const uint32_t byte = *reinterpret_cast<const uint32_t*>(c.cache + scales_at(c, cell)) >> (8 * u.group) & 0xFFu;
        const float scale = __uint_as_float(byte << 23);
        x[0] = fp4_open(codes.x, scale), x[1] = fp4_open(codes.y, scale);
        x[2] = fp4_open(codes.z, scale), x[3] = fp4_open(codes.w, scale);
        if (byte == kScaleNan)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = U32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    }
    const bool of_v = u.group >> 1;
    uint16_t* out = of_v ? v + u.l * r.v_ls + u.t * r.v_rs + u.h * r.v_hs : k + u.l * r.k_ls + u.t * r.k_rs + u.h * r.k_hs;
#pragma unroll
    for (int i = 0; i < 4; ++i) store16(out + 32 * (u.group & 1u) + 8 * i, x[i]);
}

dim3 grid_of(const Fp4Rows& r) { return dim3((uint32_t)((r.T * r.H + kThreads / 4 - 1) / (kThreads / 4)), (uint32_t)r.L); }

}  // namespace

int64_t fp4_page(int64_t block_size) { return fp4_page_bytes(block_size); }

int launch_fp4_store(const Fp4Rows& r, const Fp4Cache& c, hipStream_t stream) {
    hipLaunchKernelGGL(fp4_store_kernel, grid_of(r), dim3(kThreads), 0, stream, r, c);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_fp4_load(const Fp4Rows& r, const Fp4Cache& c, uint16_t* k, uint16_t* v, bool fill, hipStream_t stream) {
    hipLaunchKernelGGL(fp4_load_kernel, grid_of(r), dim3(kThreads), 0, stream, r, c, k, v, fill);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
