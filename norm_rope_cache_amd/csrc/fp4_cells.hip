// Rows of K and V into cells of 4 bits and back, all layers of a call in one
// launch.
//
// A group of 32 elements with the largest magnitude m gets the least power of
// two 2^e with m <= 6 2^e, so that no element saturates (e is held to -120 ..
// 125), and each element the nearest code of x / 2^e, ties to the even one. m's exponent
// and fraction say e: m = f 2^E with 1 <= f < 2 needs E - 2 up to f = 1.5, else E - 1.
// A cell with an infinity or NaN anywhere gets scale bytes of 255 and stands for NaN.
//
// Bound by memory: 256 bytes a cell on the bf16 side, 68 on the other, where a
// cell's K codes, V codes and scales are three pieces of 32, 32 and 4 bytes: tokens whose
// slots follow each other fill lines together, scattered ones cost a line each. A
// group's maximum comes by packed 16-bit maxima of the magnitudes' bits, the codes
// by the hardware's conversion, two elements a time.
#include "../../include/nrc.h"
#include "div.h"
#include "draft_ops.h"
#include "fp4.h"

namespace nrc {
namespace {

constexpr int kThreads = 256, kGroups = kThreads / 16;
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Both kernels' divisors, as products.
struct Divs {
    Div by_heads, by_block;
};
Divs divs_of(const Fp4Rows& r, const Fp4Cache& c) { return Divs{div_by((uint32_t)r.H), div_by(c.block_size)}; }

// The cell of a slot: its page's first byte in layer l's head h and its place there; false without one.
struct Cell {
    int64_t page;
    uint32_t at;
};
__device__ __forceinline__ bool cell_of(const Fp4Cache& c, Div by_block, int64_t slot, uint32_t l, uint32_t h, Cell* out) {
    if (slot < 0 || slot >= (int64_t)c.num_blocks * c.block_size) return false;
    const uint32_t block = quotient((uint32_t)slot, by_block);
    out->at = (uint32_t)slot - block * c.block_size;
    out->page = l * c.layer_stride + block * c.block_stride + h * c.head_stride;
    return true;
}
// Of a lane of the cell's 16 (8 of K, 8 of V): its dword of codes.
__device__ __forceinline__ int64_t codes_at(const Fp4Cache& c, const Cell& cell, uint32_t lane) {
    return cell.page + (int64_t)(lane >> 3) * kFp4Codes * c.block_size + cell.at * kFp4Codes + (lane & 7u) * 4;
}
__device__ __forceinline__ int64_t scales_at(const Fp4Cache& c, const Cell& cell) {
    return cell.page + 2ll * kFp4Codes * c.block_size + cell.at * 4ll;
}

// A unit: one head of one row, number `id` of a layer's (its layer: blockIdx.y).
struct Unit {
    int64_t t;
    uint32_t h;
    bool there;
};
__device__ __forceinline__ Unit unit_of(const Fp4Rows& r, Div by_heads, uint32_t id) {
    Unit u;
    u.there = id < (uint32_t)(r.T * r.H);
    u.t = u.there ? quotient(id, by_heads) : 0u;
    u.h = u.there ? id - (uint32_t)u.t * (uint32_t)r.H : 0u;
    return u;
}

// Four lanes a unit, one group of 32 elements a lane: its 64 bytes in four loads on the way together. (With 16 lanes a
// unit, 8197 rows of 8 heads in 4 layers take 25.7 us instead of 21.7: four times the lanes work out a cell's place.)
__global__ __launch_bounds__(kThreads) void fp4_store_kernel(Fp4Rows r, Fp4Cache c, Divs by) {
    const uint32_t l = blockIdx.y, group = threadIdx.x & 3u;
    const Unit u = unit_of(r, by.by_heads, blockIdx.x * (kThreads / 4) + (threadIdx.x >> 2));
    if (!u.there) return;  // (a unit's lanes go together)
    const uint16_t* src = (group >> 1 ? r.v + l * r.v_ls + u.t * r.v_rs + u.h * r.v_hs
                                      : r.k + l * r.k_ls + u.t * r.k_rs + u.h * r.k_hs) + 32 * (group & 1u);
    U32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = load16(src + 8 * i);
    Cell cell;
    if (!cell_of(c, by.by_block, r.slots[l * r.slots_ls + u.t], l, u.h, &cell)) return;
    u16x2 most{0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, (&x[i / 4].x)[i % 4] & 0x7FFF7FFFu));
    const uint32_t m = most.x > most.y ? most.x : most.y;
    // 1.5's fraction bits are 0x40; subnormals (exponent 0) end at the lowest scale
    const uint32_t down = (m & 0x7Fu) <= 0x40u ? 2u : 1u;
    uint32_t byte = m >> 7;
    byte = byte < kScaleLow + down ? kScaleLow : byte - down;
    byte = byte > kScaleHigh ? kScaleHigh : byte;
    const float scale = __uint_as_float(byte << 23);
    // the scale dword, from the cell's four groups (quad permutes); all ones for a cell with an infinity or NaN
    uint32_t bytes = m >= 0x7F80u ? 0xFFFFFFFFu : byte << (8 * group);
    bytes |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bytes, 0xB1, 0xF, 0xF, true);
    bytes |= (uint32_t)__builtin_amdgcn_mov_dpp((int)bytes, 0x4E, 0xF, 0xF, true);
    U32x4 codes{fp4_close(x[0], scale), fp4_close(x[1], scale), fp4_close(x[2], scale), fp4_close(x[3], scale)};
    if (bytes == 0xFFFFFFFFu) codes = U32x4{0u, 0u, 0u, 0u};
    store16(c.cache + codes_at(c, cell, 4 * group), codes);
    if (group == 0) *reinterpret_cast<uint32_t*>(c.cache + scales_at(c, cell)) = bytes;
}

// 16 lanes a unit, a dword of codes a lane, so that rows are written in whole runs of 128 bytes (a group a lane: 29.6
// us for what took 22.1 so; 21.1 with places by products); U units to a lane, their loads on the way together.
// fill: rows without a cell become 0, not left as they are.
template <int U>
__global__ __launch_bounds__(kThreads) void fp4_load_kernel(Fp4Rows r, Fp4Cache c, Divs by,
                                                            uint16_t* __restrict__ k, uint16_t* __restrict__ v, bool fill) {
    const uint32_t l = blockIdx.y, lane = threadIdx.x & 15u, part = lane >> 3;
    uint16_t* dst = (part ? v + l * r.v_ls : k + l * r.k_ls) + 8 * (lane & 7u);
    const int64_t rs = part ? r.v_rs : r.k_rs, hs = part ? r.v_hs : r.k_hs;
    auto id = [&](int j) { return (blockIdx.x * U + j) * kGroups + (threadIdx.x >> 4); };
    int64_t slot[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const Unit u = unit_of(r, by.by_heads, id(j));
        slot[j] = u.there ? r.slots[l * r.slots_ls + u.t] : -1;
    }
    uint32_t codes[U], bytes[U];
    bool there[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        Cell cell;
        there[j] = cell_of(c, by.by_block, slot[j], l, unit_of(r, by.by_heads, id(j)).h, &cell);
        codes[j] = bytes[j] = 0u;
        if (there[j]) {
            codes[j] = *reinterpret_cast<const uint32_t*>(c.cache + codes_at(c, cell, lane));
            bytes[j] = *reinterpret_cast<const uint32_t*>(c.cache + scales_at(c, cell));
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const Unit u = unit_of(r, by.by_heads, id(j));
        if (!u.there || (!there[j] && !fill)) continue;
        const uint32_t byte = bytes[j] >> (8 * (lane >> 2)) & 0xFFu;
        U32x4 x = there[j] ? fp4_open(codes[j], __uint_as_float(byte << 23)) : U32x4{0u, 0u, 0u, 0u};
        if (there[j] && byte == kScaleNan) x = U32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        store16(dst + u.t * rs + u.h * hs, x);
    }
}

dim3 grid_of(const Fp4Rows& r, int64_t units) { return dim3((uint32_t)((r.T * r.H + units - 1) / units), (uint32_t)r.L); }

}  // namespace

int64_t fp4_page(int64_t block_size) { return fp4_page_bytes(block_size); }

int launch_fp4_store(const Fp4Rows& r, const Fp4Cache& c, hipStream_t stream) {
    hipLaunchKernelGGL(fp4_store_kernel, grid_of(r, kThreads / 4), dim3(kThreads), 0, stream, r, c, divs_of(r, c));
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

int launch_fp4_load(const Fp4Rows& r, const Fp4Cache& c, uint16_t* k, uint16_t* v, bool fill, hipStream_t stream) {
    // (a drafting step's few rows: a unit a lane, all at once)
    if (r.T * r.H * r.L < 65536)
        hipLaunchKernelGGL(fp4_load_kernel<1>, grid_of(r, kGroups), dim3(kThreads), 0, stream, r, c, divs_of(r, c), k, v, fill);
    else
        hipLaunchKernelGGL(fp4_load_kernel<4>, grid_of(r, 4 * kGroups), dim3(kThreads), 0, stream, r, c, divs_of(r, c), k, v, fill);
    return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace nrc
