// The products of the experts' rows with their weights, both in microscaled 4-bit floating point:
//   y[r, n] = sum_h X[r, h] W_e[n, h]        for the rows r of expert e's segment, float32 sums
//   out = y, or gated (W_e's first N rows the gate, the next N the up): out[r, n] = silu(y[r, n]) * y[r, N + n]
// A matrix instruction (v_mfma_scale_f32_16x16x128) takes 16 rows of each operand by 128 elements: lane l holds the 32
// elements of block l / 16 of row l % 16, and the block's scale.
#include <algorithm>

#include "moe_common.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMxBlock = 32;
constexpr int kFp4 = 4;  // format selector of the matrix instructions
constexpr int kPlanThreads = 256;

struct ProductArgs {
    const uint8_t *x, *xs;
    const int32_t *src_row;
    const uint8_t *w, *ws;
    const int32_t *group_list, *counts;
    void *out;
    int64_t x_rows, R, H, N;
    int32_t E, capacity;
    uint32_t col_tiles;
};

// Expert e's rows, kept inside [0, R) whatever the arrays hold.
__device__ __forceinline__ void segment(const ProductArgs &a, int e, int64_t &start, int64_t &len)
{
    int64_t end;
    if (a.capacity > 0) {
        start = static_cast<int64_t>(e) * a.capacity;
        end = start + min(max(a.counts[e], 0), a.capacity);
    } else {
        start = e > 0 ? a.group_list[e - 1] : 0;
        end = a.group_list[e];
        if (a.counts)
            end = min(end, start + max(a.counts[e], 0));
    }
    start = min(max(start, int64_t{0}), a.R);
    end = min(max(end, start), a.R);
    len = end - start;
}

struct Tile {
    int32_t e;      // expert, -1: no such tile
    int32_t rows;   // rows of the tile
    int64_t first;  // its first row
};

// The m-th tile of BM rows, experts in order. Every thread of a workgroup of kPlanThreads calls it and gets the same.
template <int BM>
__device__ __forceinline__ Tile find_tile(const ProductArgs &a, int64_t m)
{
    __shared__ int64_t wave_tiles[kPlanThreads / kWave];
    __shared__ Tile found;
    constexpr int kPer = MOE_MAX_EXPERTS / kPlanThreads;
    const int per = static_cast<int>(ceil_div(a.E, kPlanThreads));
    const int e0 = threadIdx.x * per;
    int64_t tiles[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        tiles[i] = 0;
        if (i < per && e0 + i < a.E) {
            int64_t start, len;
            segment(a, e0 + i, start, len);
            tiles[i] = ceil_div(len, BM);
            mine += tiles[i];
        }
    }
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const int64_t o = __shfl_up(upto, d);
        upto += lane >= d ? o : 0;
    }
    if (lane == kWave - 1)
        wave_tiles[wave] = upto;
    if (threadIdx.x == 0)
        found = Tile{-1, 0, 0};
    __syncthreads();
    int64_t before = upto - mine;
    for (int v = 0; v < wave; ++v)
        before += wave_tiles[v];
    if (m >= before && m < before + mine) {
        int64_t k = m - before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (k >= 0 && k < tiles[i]) {
                int64_t start, len;
                segment(a, e0 + i, start, len);
                found = Tile{e0 + i, static_cast<int32_t>(min(len - k * BM, int64_t{BM})), start + k * BM};
            }
            k -= tiles[i];
        }
    }
    __syncthreads();
    return found;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t *p, float v) { *p = static_cast<uint16_t>(f32_to_bf16_bits(v)); }

// A lane's block of a row: zeros where there is none (block >= blocks or no row).
__device__ __forceinline__ void load_block(const uint8_t *codes, const uint8_t *scales, int64_t row, int64_t blocks, int64_t b,
                                           bool there, i32x8 &v, int &scale)
{
    u32x4 c{0, 0, 0, 0};
    scale = 127;
    if (there && b < blocks) {
        c = ld16(codes + (row * blocks + b) * 16);
        scale = scales[row * blocks + b];
    }
    v = i32x8{static_cast<int>(c.x), static_cast<int>(c.y), static_cast<int>(c.z), static_cast<int>(c.w), 0, 0, 0, 0};
}

// Four wavefronts a workgroup, each a tile of 16 rows by 16 columns.
template <typename O, bool GATED>
__global__ __launch_bounds__(kPlanThreads) void grouped_product_kernel(ProductArgs a)
{
    const Tile tile = find_tile<16>(a, blockIdx.x / a.col_tiles);
    if (tile.e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
    const int64_t n0 = (static_cast<int64_t>(blockIdx.x % a.col_tiles) * (kPlanThreads / kWave) + threadIdx.x / kWave) * 16;
    if (n0 >= a.N)
        return;
    const int64_t blocks = a.H / kMxBlock;
    int64_t row = tile.first + min(r, tile.rows - 1);
    bool there = r < tile.rows;
    if (a.src_row) {
        row = a.src_row[row];
        there = there && row >= 0 && row < a.x_rows;
        row = there ? row : 0;
    }
    const int64_t n = n0 + r, wrows = a.N * (GATED ? 2 : 1), wrow = tile.e * wrows + n;
    f32x4 acc{0, 0, 0, 0}, up{0, 0, 0, 0};
    for (int64_t b = g; b < blocks + g; b += 4) {
        i32x8 vx, vw;
        int sx, sw;
        load_block(a.x, a.xs, row, blocks, b, there, vx, sx);
        load_block(a.w, a.ws, wrow, blocks, b, n < a.N, vw, sw);
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vx, vw, acc, kFp4, kFp4, 0, sx, 0, sw);
        if constexpr (GATED) {
            load_block(a.w, a.ws, wrow + a.N, blocks, b, n < a.N, vw, sw);
            up = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vx, vw, up, kFp4, kFp4, 0, sx, 0, sw);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = 4 * g + i;
        if (m < tile.rows && n < a.N)
            store_out(static_cast<O *>(a.out) + (tile.first + m) * a.N + n, GATED ? silu(acc[i]) * up[i] : acc[i]);
    }
}

// Tiles of BM rows that R rows in E segments can need.
int64_t max_tiles(int64_t R, int64_t E, int64_t BM) { return R / BM + std::min(R, E); }

template <typename O, bool GATED>
moe_status launch_product(ProductArgs a, hipStream_t stream)
{
    a.col_tiles = static_cast<uint32_t>(ceil_div(a.N, 16 * (kPlanThreads / kWave)));
    const int64_t grid = max_tiles(a.R, a.E, 16) * a.col_tiles;
    if (grid > 0x7fffffff)
        return MOE_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((grouped_product_kernel<O, GATED>), dim3(static_cast<unsigned>(grid)), dim3(kPlanThreads), 0, stream, a);
    return launch_status();
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_grouped_product_mxfp4(const uint8_t *x, const uint8_t *x_scales, int64_t x_rows,
                                                const int32_t *src_row, int64_t R, int64_t H, const uint8_t *w,
                                                const uint8_t *w_scales, int32_t E, int64_t N, int32_t gated,
                                                const int32_t *group_list, const int32_t *counts, int32_t capacity, void *out,
                                                moe_dtype out_dt, hipStream_t stream)
{
    using namespace moe;
    if (R < 0 || x_rows < 0 || H < 1 || H % kMxBlock != 0 || N < 1 || E < 1 || capacity < 0 ||
        (out_dt != MOE_F32 && out_dt != MOE_BF16 && out_dt != MOE_FP8_E4M3) || (!src_row && x_rows < R) ||
        (capacity > 0 && R < static_cast<int64_t>(E) * capacity))
        return MOE_ERR_INVALID;
    if (out_dt == MOE_FP8_E4M3 || E > MOE_MAX_EXPERTS || R > 0x7fffffff || x_rows > 0x7fffffff || H > (1 << 20) || N > (1 << 20))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0)
        return MOE_OK;
    if ((x_rows > 0 && (!x || !x_scales)) || !w || !w_scales || !out || (capacity > 0 ? !counts : !group_list))
        return MOE_ERR_INVALID;
    if (!aligned16(x) || !aligned16(w))
        return MOE_ERR_UNSUPPORTED;
    const ProductArgs a{x, x_scales, src_row, w, w_scales, group_list, counts, out, x_rows, R, H, N, E, capacity, 0};
    if (out_dt == MOE_F32)
        return gated ? launch_product<float, true>(a, stream) : launch_product<float, false>(a, stream);
    return gated ? launch_product<uint16_t, true>(a, stream) : launch_product<uint16_t, false>(a, stream);
}
