// The products of the experts' rows with their weights, both in microscaled 4-bit floating point:
//   y[r, n] = sum_h X[r, h] W_e[n, h]        for the rows r of expert e's segment, float32 sums
//   out = y, or gated (W_e's first N rows the gate, the next N the up): out[r, n] = silu(y[r, n]) * y[r, N + n]
// The matrix instructions take both operands' codes with their scales: of 16x16x128 lane l holds the 32 elements of block l / 16 of
// row l % 16, of 32x32x64 those of block l / 32 of row l % 32, and the block's scale byte. The weights are the first operand, so
// that a lane's sums are of consecutive columns. An expert with few rows is bound by reading its weights, one with many by the
// matrix instructions (6.7 PFLOP/s is what they reach by themselves here with random codes, at 1.66 GHz; with zeros, whose products
// take less power, 9.8 at 2.39 GHz); there is a kernel for each. Both sum over h in the order of the elements, or in four parts of it.
#include <algorithm>
#include <type_traits>

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

// A workgroup's share: columns from `col` tiles on, of `rows` rows from `first` on, of expert e.
struct Tile {
    int32_t e;      // -1: none
    int32_t rows;
    int64_t first;
    int32_t col;
};

// The i-th of the (rows, columns) tiles of BM rows: experts in order, of an expert kGroup tiles of the same columns beside each
// other. (Those that run at the same time on an XCD then share both their weights and their rows in its L2: one expert of 8192
// cubed 334 -> 298 us against all the rows' tiles first.) Every thread of a workgroup of kPlanThreads calls it and gets the same.
// Of up to four tiles of 256 the rows are dealt out evenly, by 32, where rows are long: two of 150 take less than one of 256 and
// one of 44 (R131072 E256 H7168 N1024 gated 1363 -> 1315 us; where they are short each tile's begin and end count more: H1024
// N7168 1077 -> 1134).
// Sums of tiles stop at 2^32 - 1, which only segments that overlap reach: no two experts then claim the i-th, i < 2^31.
constexpr uint32_t kGroup = 8;
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

struct Search {
    Tile found;
    uint32_t wave_tiles[kPlanThreads / kWave];
};

template <int BM>
__device__ __forceinline__ Tile find_tile(const ProductArgs &a, uint32_t i, Search &sh)
{
    uint32_t *const wave_tiles = sh.wave_tiles;
    Tile &found = sh.found;
    constexpr int kPer = MOE_MAX_EXPERTS / kPlanThreads;
    const int per = static_cast<int>((a.E + kPlanThreads - 1) / kPlanThreads), e0 = threadIdx.x * per;
    uint32_t tiles[kPer], start[kPer], len[kPer], height[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        tiles[j] = start[j] = len[j] = height[j] = 0;
        if (j < per && e0 + j < a.E) {
            int64_t s, l;
            segment(a, e0 + j, s, l);
            start[j] = static_cast<uint32_t>(s);
            len[j] = static_cast<uint32_t>(l);
            const uint32_t n = (len[j] + BM - 1) / BM;
            height[j] = BM == 256 && a.H >= 2048 && n > 1 && n <= 4 ? ((len[j] + n - 1) / n + 31) / 32 * 32 : BM;
            tiles[j] = n * a.col_tiles;
            mine = add_sat(mine, tiles[j]);
        }
    }
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t o = __shfl_up(upto, d);
        upto = add_sat(upto, lane >= d ? o : 0);
    }
    if (lane == kWave - 1)
        wave_tiles[wave] = upto;
    if (threadIdx.x == 0)
        found = Tile{-1, 0, 0, 0};
    uint32_t before = __shfl_up(upto, 1);
    before = lane == 0 ? 0 : before;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kPlanThreads / kWave - 1; ++v)
        before = add_sat(before, v < wave ? wave_tiles[v] : 0);
    if (i >= before && i - before < mine) {
        uint32_t k = i - before;
        bool left = true;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (left && k < tiles[j]) {
                left = false;
                const uint32_t n = (len[j] + BM - 1) / BM, g = k / (kGroup * a.col_tiles), in = k % (kGroup * a.col_tiles);
                const uint32_t high = min(kGroup, n - kGroup * g), m = kGroup * g + in % high;
                found = Tile{e0 + j, static_cast<int32_t>(min(len[j] - m * height[j], height[j])),
                             static_cast<int64_t>(start[j]) + m * height[j], static_cast<int32_t>(in / high)};
            }
            k -= tiles[j];
        }
    }
    __syncthreads();
    // one for the wavefront: into scalar registers
    const int64_t first = found.first;
    return Tile{__builtin_amdgcn_readfirstlane(found.e), __builtin_amdgcn_readfirstlane(found.rows),
                static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(first >> 32))) << 32 |
                    static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(first))),
                __builtin_amdgcn_readfirstlane(found.col)};
}

// g / (1 + exp(-g)) by the instructions for 2^x and 1 / x, right to an ulp each: with the argument's rounding (|g| + 6) u in all.
// (log2 e alone is off by 0.23 u of itself, which would be |g| 0.23 u more: its low part goes into the same rounding.)
// 1 / x gives 0 for results below the normal numbers, as 1 / (1 + exp(-g)) is from g = -87.3 on: it is taken of a sixteenth, and
// the product with 1/16 keeps 21 bits or more there (4 u besides). Past g = -88.72 exp(-g) passes float32: 0.
__device__ __forceinline__ float silu(float g)
{
    constexpr float kLog2e = 1.44269504088896340736f, kLow = 1.925963033500e-8f;  // their sum is log2 e
    constexpr float kPart = 1.0f / 16;
    const float e = __builtin_amdgcn_exp2f(fmaf(-kLog2e, g, -kLow * g));
    return g * (__builtin_amdgcn_rcpf(fmaf(e, kPart, kPart)) * kPart);
}

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t *p, float v) { *p = static_cast<uint16_t>(f32_to_bf16_bits(v)); }

// Four values to consecutive places.
__device__ __forceinline__ void put4(float *p, const float (&v)[4]) { *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ void put4(uint16_t *p, const float (&v)[4])
{
    *reinterpret_cast<uint64_t *>(p) = pack_bf16x2(v[0], v[1]) | static_cast<uint64_t>(pack_bf16x2(v[2], v[3])) << 32;
}

// ---------------------------------------------------------------- few rows an expert

// The bytes of v from byte n (< 16) on, zeros behind them.
__device__ __forceinline__ u32x4 shifted(const u32x4 &v, int n)
{
    const uint32_t w0 = n & 8 ? v.z : v.x, w1 = n & 8 ? v.w : v.y, w2 = n & 8 ? 0 : v.z, w3 = n & 8 ? 0 : v.w;
    const uint32_t u0 = n & 4 ? w1 : w0, u1 = n & 4 ? w2 : w1, u2 = n & 4 ? w3 : w2, u3 = n & 4 ? 0 : w3;
    return u32x4{__builtin_amdgcn_alignbyte(u1, u0, n), __builtin_amdgcn_alignbyte(u2, u1, n),
                 __builtin_amdgcn_alignbyte(u3, u2, n), __builtin_amdgcn_alignbyte(0, u3, n)};
}

// The scale bytes of a row of fewer than 16 blocks.
__device__ __forceinline__ u32x4 short_scales(const uint8_t *row, int blocks)
{
    uint64_t w[2] = {0, 0};
    for (int i = 0; i < blocks; ++i)
        w[i / 8] |= static_cast<uint64_t>(row[i]) << (8 * (i % 8));
    return u32x4{static_cast<uint32_t>(w[0]), static_cast<uint32_t>(w[0] >> 32), static_cast<uint32_t>(w[1]),
                 static_cast<uint32_t>(w[1] >> 32)};
}

constexpr int kRunBytes = 256, kRunBlocks = kRunBytes / 16;  // of each row at a time: 512 elements, 16 scale bytes
constexpr int kDppRowRor8 = 0x128;
constexpr int kRowsWorkgroups = 3;  // a CU: their registers are 168 a thread

// Weights come in whole cache lines: an instruction reads 128 bytes of 8 rows, rows 0..7 into a and 8..15 into b, lanes 8..15 of
// each 16 the second 64 bytes. Swapping lanes 8..15 of a with 0..7 of b leaves the two 64-byte halves of all 16 rows.
__device__ __forceinline__ void swap_eights(uint32_t &a, uint32_t &b)
{
    const int x = static_cast<int>(a), y = static_cast<int>(b);
    a = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(x, y, kDppRowRor8, 0xf, 0xc, false));
    b = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(y, x, kDppRowRor8, 0xf, 0x3, false));
}

__device__ __forceinline__ i32x8 operand(const u32x4 &v)
{
    return i32x8{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w), 0, 0, 0, 0};
}

// A wavefront's share of 512 elements: 32 weight rows and 16 rows of x, with their scales.
struct Weights {
    u32x4 v[2][4], scales[2];
};
struct Rows {
    u32x4 v[4], scales;
};

// Up to 16 rows of an expert by 32 weight rows (gated: 16 of the gate and the 16 of the up of the same columns) a wavefront. The
// weights go from memory into the matrix instructions' operand registers, the next 512 elements on their way while these are
// multiplied. SPLIT wavefronts share the columns and take parts of the sum, put together in LDS.
// Bound by reading the weights: 512 rows of E128 H2048 N4096, 570 MB in 92 us (6.2 TB/s; a large read reaches 6.7); one token's 8
// experts of E256 H7168 N1024 gated, 62 MB in 12.7 (4.9), of which the search of the segment, the first loads and the last are 4.
// The weights through the caches' streaming policy and in whole lines; x's rows are single buffered, so that three workgroups fit a
// CU (double buffered, two of them: 110 us).
template <typename O, bool GATED, int SPLIT>
__global__ __launch_bounds__(kPlanThreads, kRowsWorkgroups) void grouped_rows_kernel(ProductArgs a)
{
    constexpr int kWaves = kPlanThreads / kWave, kCols = GATED ? 16 : 32;  // columns of a wavefront
    __shared__ f32x4 sums[SPLIT > 1 ? kWaves : 1][2][kWave];
    __shared__ Search search;
    const Tile tile = find_tile<16>(a, blockIdx.x, search);
    if (tile.e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / kWave));
    const int r = lane & 15, g = lane >> 4, part = wave % SPLIT;
    const int64_t n0 = (static_cast<int64_t>(tile.col) * (kWaves / SPLIT) + wave / SPLIT) * kCols;
    const int blocks = static_cast<int>(a.H / kMxBlock), runs = (blocks + kRunBlocks - 1) / kRunBlocks;
    const int64_t wrows = a.N * (GATED ? 2 : 1);
    const uint32_t row_bytes = static_cast<uint32_t>(a.H / 2);
    const int cols = static_cast<int>(min(a.N - n0, static_cast<int64_t>(kCols)));  // this wavefront's, if any
    f32x4 acc[2] = {};

    // lane l holds row l % 16 and four consecutive columns of each 16
    O *const out = static_cast<O *>(a.out) + (tile.first + r) * a.N + n0;
    const bool vectors = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & (4 * sizeof(O) - 1)) == 0;
    auto store = [&]() {
        if (r < tile.rows) {
#pragma unroll
            for (int i = 0; i < (GATED ? 1 : 2); ++i) {
                const int c = 16 * i + 4 * g;
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = GATED ? silu(acc[0][q]) * acc[1][q] : acc[i][q];
                if (vectors) {
                    if (c < cols)
                        put4(out + c, v);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (c + q < cols)
                            store_out(out + c + q, v[q]);
                }
            }
        }
    };

    if (cols > 0) {
        int64_t row = tile.first + min(r, tile.rows - 1);  // x's row r
        bool there = r < tile.rows;
        if (a.src_row) {
            row = a.src_row[row];
            there = there && row >= 0 && row < a.x_rows;
            row = there ? row : 0;
        }
        const uint8_t *const x = a.x + row * row_bytes, *const xs = there ? a.xs + row * blocks : a.ws;
        // weights from this wavefront's first column on (gated: of the gate and of the up)
        const int64_t at = tile.e * wrows + n0;
        const uint8_t *ws[2];
        __amdgpu_buffer_rsrc_t wr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t first = at + (GATED ? i * a.N : 0);
            wr[i] = make_rsrc(a.w + first * row_bytes,
                              static_cast<uint32_t>(min((a.E * wrows - first) * row_bytes, static_cast<int64_t>(0xfffffff0))));
            ws[i] = a.ws + first * blocks;
        }
        auto scales = [&](const uint8_t *from, int run) -> u32x4 {
            if (blocks < kRunBlocks)
                return short_scales(from, blocks);
            u32x4 v;
            __builtin_memcpy(&v, from + min(run * kRunBlocks, blocks - kRunBlocks), sizeof(v));
            return v;
        };
        auto load_w = [&](int run, Weights &to) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = GATED ? 0 : 16 * i;  // past the last column that column's weights
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t o = min(n + 8 * j + (r & 7), cols - 1) * row_bytes + (g + (r & 8) / 2) * 16 + run * kRunBytes;
                    to.v[i][j] = ld16_buf<kPolicyStreamLoad>(wr[i], o);
                    to.v[i][2 + j] = ld16_buf<kPolicyStreamLoad>(wr[i], o + 128);
                }
                to.scales[i] = scales(ws[i] + min(n + r, cols - 1) * blocks, run);
            }
        };
        auto load_x = [&](int run, Rows &to) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int b = run * kRunBlocks + 4 * j + g;
                to.v[j] = u32x4{0, 0, 0, 0};
                if (there && b < blocks)
                    to.v[j] = ld16(x + b * 16);
            }
            to.scales = scales(xs, run);
        };
        const uint32_t keep = there ? 0xffffffffu : 0;  // beside zeros the scale is any but NaN
        auto multiply = [&](int run, Weights &w, const Rows &x) {
            const int past = blocks < kRunBlocks ? 0 : run * kRunBlocks - min(run * kRunBlocks, blocks - kRunBlocks);
            const u32x4 sx = shifted(x.scales, past);
            const uint32_t s[4] = {sx.x & keep, sx.y & keep, sx.z & keep, sx.w & keep};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x4 sw = shifted(w.scales[i], past);
                const uint32_t t[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    u32x4 &p = w.v[i][j], &q = w.v[i][j + 1];
                    swap_eights(p.x, q.x);
                    swap_eights(p.y, q.y);
                    swap_eights(p.z, q.z);
                    swap_eights(p.w, q.w);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        operand(w.v[i][j]), operand(x.v[j]), acc[i], kFp4, kFp4, 0, static_cast<int>(t[j] >> (8 * g)), 0,
                        static_cast<int>(s[j] >> (8 * g)));
            }
        };
        const int from = runs * part / SPLIT, to = runs * (part + 1) / SPLIT;
        if (from < to) {
            Weights f[2];
            Rows rows;
            load_w(from, f[0]);
            load_x(from, rows);
            int run = from;
            for (; run + 2 < to; run += 2) {
                load_w(run + 1, f[1]);
                multiply(run, f[0], rows);
                load_x(run + 1, rows);
                load_w(run + 2, f[0]);
                multiply(run + 1, f[1], rows);
                load_x(run + 2, rows);
            }
            if (run + 1 < to) {
                load_w(run + 1, f[1]);
                multiply(run, f[0], rows);
                load_x(run + 1, rows);
                multiply(run + 1, f[1], rows);
            } else {
                multiply(run, f[0], rows);
            }
        }
    }
    if constexpr (SPLIT > 1) {
        if (part > 0) {
            sums[wave][0][lane] = acc[0];
            sums[wave][1][lane] = acc[1];
        }
        __syncthreads();
        if (part > 0)
            return;
#pragma unroll
        for (int p = 1; p < SPLIT; ++p) {
            acc[0] += sums[wave + p][0][lane];
            acc[1] += sums[wave + p][1][lane];
        }
    }
    if (cols > 0)
        store();
}

// ---------------------------------------------------------------- tiles through LDS

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kStageBytes = 64;                  // of each row a stage: 128 elements
constexpr int kStageBlocks = kStageBytes / 16;
constexpr int kStages = 4;                       // of which LDS has room
constexpr int kScaleStages = 4;                  // stages whose scales come at a time: 16 bytes of a row
constexpr int kLineStages = 8;                   // or 32 bytes, where rows of scales begin at multiples of 16 bytes

// The 16-byte chunk c of row r lies in slot c ^ swizzle(r) of its 64 bytes: 8 and 16 consecutive rows' same chunk fall into
// different banks.
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); }

template <int ROWS, int COLS, bool LINES>
struct Buffers {
    uint8_t codes[kStages][(ROWS + COLS) * kStageBytes];
    uint32_t scales[2][ROWS + COLS][LINES ? kLineStages : kScaleStages];
};

// 16 bytes a lane into LDS, lane l's to address `to` + 16 l (one for the wavefront). Past the resource's end: zeros.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, uint32_t to)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, reinterpret_cast<__attribute__((address_space(3))) void *>(to), 16,
                                             static_cast<int>(offset), 0, 0, 0);
}

// The same by an address of each lane's.
__device__ __forceinline__ void to_lds(const uint8_t *from, uint32_t to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     reinterpret_cast<__attribute__((address_space(3))) void *>(to), 16, 0, 0);
}

__device__ const u32x4 kZeros = {0, 0, 0, 0};  // what such a load reads of a row that is not there

// Buffer resources end before this offset, which asks for nothing.
constexpr uint32_t kNowhere = 0xfffffff0u;

__device__ __forceinline__ uint32_t capped(int64_t bytes)
{
    return static_cast<uint32_t>(min(bytes, static_cast<int64_t>(kNowhere)));
}

template <int MS, int NS>
struct Frags {
    i32x8 x[MS], w[NS];
};

// Workgroup b of nb, dealt to the XCDs in turn, takes the place that keeps runs of kRun neighbours on one XCD.
constexpr uint32_t kRun = 16;
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t nb)
{
    const uint32_t round = b / (kXcds * kRun), in = b % (kXcds * kRun);
    return (round + 1) * kXcds * kRun > nb ? b : round * kXcds * kRun + in % kXcds * kRun + in / kXcds;
}

// A tile of up to ROWS rows by COLS weight rows (gated: half of the gate and the half of the up of the same columns), four
// wavefronts. Wide tiles are 256 by 256: of more than 128 rows a wavefront has 128 by 128 weight rows, two wavefronts beside each
// other each way; of fewer all of them by 64 weight rows. Tiles of 128 by 128, a wavefront with 64 by 64 or, of up to 64 rows, 32
// by 64, two to a CU, are for products of which the wide ones would leave CUs without one. Gated, a wavefront's first half are
// gates, its second the ups of the same columns.
// A product's operands are read from LDS a step ahead, and stages of 128 elements come three ahead by loads that write LDS
// themselves; what is issued between two products is spread out by the scheduling barriers. R131072 E256 H7168 N1024 gated with
// a map 1.17-1.24 ms (3.85e12 operations, 3.1-3.3 PFLOP/s), 8192 cubed 265 us (4.1). There a stage takes 1466 cycles (at 1.67 GHz, the
// power's limit), 1295 without its loads (at 1.91), of which the matrix instructions by themselves are 1036: bound by them, by
// what feeds them and by the power, and by each tile's begin and end (search and first stages 4-5 us, outputs 3-4), when its CU has
// nothing else to do: R131072 E256 H1024 N7168 1.00-1.05 ms (1.9 PFLOP/s; its outputs alone are 1.9 GB).
// FAR is for a map onto more codes than a buffer resource's 32-bit offsets reach: x comes by 64-bit addresses (R131072 E256 H7168
// N1024 gated of 1.2 M rows 1.53 ms, of 1.19 M by offsets 1.30; 16 rows a workgroup without tiles took 12.4).
template <typename O, bool GATED, int ROWS, int COLS, bool LINES, bool FAR>
__global__ __launch_bounds__(kPlanThreads) void grouped_tile_kernel(ProductArgs a)
{
    constexpr bool kWide = COLS == 256;
    static_assert(ROWS == COLS && (kWide || COLS == 128), "");
    __shared__ __attribute__((aligned(128))) Buffers<ROWS, COLS, LINES> sh;  // wide, with lines: all of a CU's LDS
    const Tile tile = find_tile<ROWS>(a, xcd_run(blockIdx.x, gridDim.x), *reinterpret_cast<Search *>(sh.scales[1]));
    if (tile.e < 0)
        return;
    __syncthreads();  // the search is done with its place
    constexpr int kOutCols = GATED ? COLS / 2 : COLS, kXMost = ROWS / 64, kWLoads = COLS / 64;  // 16-byte loads a thread and stage
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / kWave));
    const int blocks = static_cast<int>(a.H / kMxBlock), stages = (blocks + kStageBlocks - 1) / kStageBlocks;
    const int64_t row_bytes = a.H / 2, n0 = static_cast<int64_t>(tile.col) * kOutCols;
    const bool big = kWide && tile.rows > 128;
    const int wave_cols = big ? 128 : 64, wave_half = wave_cols / 2;

    // A load takes 16 rows a wavefront, 4 lanes a row: thread t chunk slot t % 4 of rows 64 j + t / 4. Loads go by buffer resources,
    // whose bounds keep what lies past the last row's end unread. x is from its tile's first row on, or whole with a map; rows that
    // are not there load zeros. The weight row, from n0 on, behind row b of the tile's weights is w_row(b), of the up if is_up(b).
    const int chunk = (lane & 3) ^ swizzle(lane >> 2);
    const int64_t x_at = a.src_row ? 0 : tile.first;
    const uint8_t *const xbase = a.x + x_at * row_bytes;
    const uint32_t xbytes = capped((a.x_rows - x_at) * row_bytes);
    const int64_t wrows = a.N * (GATED ? 2 : 1), w_at = tile.e * wrows + n0;
    // (without a map some number that is there, and not used: the loads need no branch and come together)
    const int32_t *const map = a.src_row ? a.src_row + tile.first : a.capacity > 0 ? a.counts : a.group_list;
    const int map_last = a.src_row ? tile.rows - 1 : 0;
    auto mapped = [&](int r) -> int32_t { return map[min(r, map_last)]; };
    // x's row r of the tile, behind the base above; -1 if there is none
    auto x_row = [&](int r, int32_t from) -> int32_t {
        const int32_t row = a.src_row ? from : r;
        return r < tile.rows && row < a.x_rows - x_at ? row : -1;
    };
    auto w_row = [&](int b) -> int32_t {
        const int n = GATED ? b / wave_cols * wave_half + b % wave_half : b;
        return min(n, static_cast<int>(a.N - 1 - n0));
    };
    auto is_up = [&](int b) { return GATED && b % wave_cols >= wave_half; };
    const int x_mine = threadIdx.x % ROWS, w_mine = threadIdx.x % COLS;  // rows whose scales a thread takes (some twice)
    // The map's entries on their way first, behind them the weights of stages 0 and 1 (R131072 E256 H7168 N1024 gated 1231 -> 1190 us,
    // H1024 N7168 1062 -> 1025, against the map's entries one by one and then all loads).
    int32_t from[kXMost], from_mine = 0, from_lines[2];
#pragma unroll
    for (int j = 0; j < kXMost; ++j)
        from[j] = mapped(64 * j + threadIdx.x / 4);
    if constexpr (LINES) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            from_lines[q] = mapped(32 * (4 * q + wave) + lane / 2);
    } else {
        from_mine = mapped(x_mine);
    }
    // where x's chunks are: by offsets, or by addresses
    std::conditional_t<FAR, const uint8_t *, uint32_t> xo[kXMost];
    uint32_t wo[kWLoads];
#pragma unroll
    for (int j = 0; j < kWLoads; ++j)
        wo[j] = static_cast<uint32_t>(w_row(64 * j + threadIdx.x / 4)) * static_cast<uint32_t>(row_bytes) + chunk * 16;
    const uint8_t *const wsp = a.ws + (w_at + w_row(w_mine) + (is_up(w_mine) ? a.N : 0)) * blocks;
    const uint8_t *const gate = a.w + w_at * row_bytes, *const up = gate + (GATED ? a.N * row_bytes : 0);
    const uint32_t gate_bytes = capped((a.E * wrows - w_at) * row_bytes);
    const uint32_t up_bytes = GATED ? capped((a.E * wrows - w_at - a.N) * row_bytes) : gate_bytes;

    // The stages' addresses as plain numbers: of what it sees to lie in the array the compiler would wait for every load under
    // way into it, those of later stages included, before each read. What a read needs has come by `meet`.
    uint32_t codes = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)&sh.codes[0][0]));
    asm volatile("" : "+s"(codes));
    auto slot = [&](int s) -> uint32_t {
        return codes + (s % kStages) * static_cast<uint32_t>(sizeof(sh.codes[0])) + wave * 16 * kStageBytes;
    };
    // x's chunks past the end of the rows are zeros (beside them the weights' are some codes, and zero times them is zero); past the
    // last stage nothing is read, but the number of loads is the same in every stage.
    auto load_x = [&](int s, int j) {
        if constexpr (FAR)
            to_lds(s * kStageBlocks + chunk < blocks && xo[j] ? xo[j] + s * kStageBytes : reinterpret_cast<const uint8_t *>(&kZeros),
                   slot(s) + 64 * j * kStageBytes);
        else
            to_lds(make_rsrc(xbase, xbytes), s * kStageBlocks + chunk < blocks && xo[j] != kNowhere ? xo[j] + s * kStageBytes : kNowhere,
                   slot(s) + 64 * j * kStageBytes);
    };
    auto load_w = [&](int s, int j) {
        const bool u = is_up(64 * j + 16 * wave);
        const uint32_t bytes = u ? up_bytes : gate_bytes;
        to_lds(make_rsrc(u ? up : gate, s < stages ? bytes : 0), wo[j] + s * kStageBytes, slot(s) + (ROWS + 64 * j) * kStageBytes);
    };
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            load_w(s, j);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kXMost; ++j) {
        const int32_t row = x_row(64 * j + threadIdx.x / 4, from[j]);
        if constexpr (FAR)
            xo[j] = row >= 0 ? xbase + row * row_bytes + chunk * 16 : nullptr;
        else
            xo[j] = row >= 0 ? static_cast<uint32_t>(row) * static_cast<uint32_t>(row_bytes) + chunk * 16 : kNowhere;
    }
    const int32_t xs_row = x_row(x_mine, from_mine);
    const uint8_t *const xsp = xs_row >= 0 ? a.xs + (x_at + xs_row) * blocks : wsp;
    const uint32_t keep = xs_row >= 0 ? 0xffffffffu : 0;  // beside zeros the scale is any but NaN
    // Scales come for kScaleStages stages (a group) at a time, x's and the weights' in turns. A row's 16 bytes are put down as what
    // each half of a wavefront needs of them: blocks 0, 1 of each stage's four, then blocks 2, 3.
    const uint8_t *const xsl = blocks >= 16 ? xsp : a.w;  // (16 bytes to read, where the rows are shorter)
    const int64_t to_wsl = blocks >= 16 ? wsp - xsp : 0;
    u32x4 sc;
    auto scale_at = [&](int g) { return max(min(16 * g, blocks - 16), 0); };  // past the end: what nothing uses
    auto load_sc = [&](bool w, int g) { __builtin_memcpy(&sc, xsl + (w ? to_wsl : 0) + scale_at(g), sizeof(sc)); };
    auto put_sc = [&](bool w, int g, const u32x4 &v) {
        const uint32_t k = w ? 0xffffffffu : keep;
        st16(sh.scales[g & 1][w ? ROWS + w_mine : x_mine],
             u32x4{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u) & k, __builtin_amdgcn_perm(v.w, v.z, 0x05040100u) & k,
                   __builtin_amdgcn_perm(v.y, v.x, 0x07060302u) & k, __builtin_amdgcn_perm(v.w, v.z, 0x07060302u) & k});
    };
    auto store_sc = [&](bool w, int g) { put_sc(w, g, shifted(sc, min(16 * g - scale_at(g), 15))); };
    // With lines they come for kLineStages stages, straight into LDS as they lie, two lanes a row: half the requests of the way above,
    // and nothing to move (R131072 E256 H7168 N1024 gated 1342 -> 1218 us, R12288 E128 251 -> 236; short of rows, H4096 E64, 32 rows an
    // expert, 117 -> 123). The loads of a group are four quarters, each 32 rows a wavefront, of which lane l has row l / 2: rows
    // 32 (4 q + wavefront) on of x's and the weights'.
    uint32_t so[4];
    uint32_t scales_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint32_t *)&sh.scales[0][0][0]));
    const bool line_up = is_up(32 * wave);
    const uint8_t *const x_lines = a.xs + x_at * blocks, *const w_lines = a.ws + (w_at + (line_up ? a.N : 0)) * blocks;
    const uint32_t x_line_bytes = capped((a.x_rows - x_at) * blocks);
    const uint32_t w_line_bytes = capped((a.E * wrows - w_at - (line_up ? a.N : 0)) * blocks);
    if constexpr (LINES) {
        asm volatile("" : "+s"(scales_at));  // (as for codes)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int b = 32 * (4 * q + wave) + lane / 2;
            const int32_t row = q < 2 ? x_row(b, from_lines[q & 1]) : w_row(b - ROWS);
            so[q] = row >= 0 ? static_cast<uint32_t>(row) * static_cast<uint32_t>(blocks) + lane % 2 * 16 : kNowhere;
        }
    }
    auto load_line = [&](int g, int q) {
        uint32_t from = 0;  // so[q], without a branch
#pragma unroll
        for (int i = 0; i < 4; ++i)
            from |= so[i] & (q == i ? 0xffffffffu : 0);
        to_lds(make_rsrc(q < 2 ? x_lines : w_lines, q < 2 ? x_line_bytes : w_line_bytes),
               from == kNowhere ? kNowhere : from + g * 4 * kLineStages,
               scales_at + (g & 1) * static_cast<uint32_t>(sizeof(sh.scales[0])) + (4 * q + wave) * 32 * 4 * kLineStages);
    };
    const auto i1 = std::integral_constant<int, 1>{};
    const auto i2 = std::integral_constant<int, 2>{};
    const auto i3 = std::integral_constant<int, 3>{};
    const auto i4 = std::integral_constant<int, 4>{};

    const int half = lane >> 5, r32 = lane & 31, swz = swizzle(r32);
    f32x16 acc[4][4];
    // The products, for tiles of up to 32 MS WM rows, WM wavefronts beside each other along the rows: a wavefront has 32 MS rows by
    // 32 NS weight rows, in acc[0 .. NS - 1], or of two, gated, in acc[0] and acc[2].
    auto products = [&](auto ms, auto ns, auto wm) {
        constexpr int MS = ms, NS = ns, WM = wm;
        static_assert(32 * NS * (4 / WM) == COLS, "");
        constexpr int kXLoads = MS * WM < 2 ? 1 : MS * WM / 2, kLoads = kXLoads + kWLoads, kStep = GATED ? 4 / NS : 1;
        const int x0 = (wave % WM) * 32 * MS + r32, w0 = ROWS + (wave / WM) * 32 * NS + r32;
        // a lane's 16 bytes in steps 0 and 1 of a stage: chunks 2 half and 2 half + 1
        const uint32_t lane_at[2] = {codes + x0 * kStageBytes + ((2 * half) ^ swz) * 16,
                                     codes + x0 * kStageBytes + ((2 * half + 1) ^ swz) * 16};
        auto frag = [&](int s, int row, int ks) -> i32x8 {
            const uint32_t at = lane_at[ks] + (s % kStages) * static_cast<uint32_t>(sizeof(sh.codes[0])) + row * kStageBytes;
            const i32x4 v = *reinterpret_cast<const __attribute__((address_space(3))) i32x4 *>(at);
            return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
        };
        Frags<MS, NS> f[2];
        auto read = [&](int s, int ks, Frags<MS, NS> &to) {
#pragma unroll
            for (int m = 0; m < MS; ++m)
                to.x[m] = frag(s, 32 * m, ks);
#pragma unroll
            for (int n = 0; n < NS; ++n)
                to.w[n] = frag(s, w0 - x0 + 32 * n, ks);
        };
        // Scales of stages s and s + 1, s even: steps 0 to 3 have bytes 0 to 3.
        int xs[MS], ws[NS], next_xs[MS], next_ws[NS];
        auto read_scale = [&](int s, int row) -> int {
            if constexpr (LINES) {
                const uint32_t at = scales_at + (s / kLineStages & 1) * static_cast<uint32_t>(sizeof(sh.scales[0])) +
                                    row * 4 * kLineStages + s % kLineStages * 4;
                const uint64_t v = *reinterpret_cast<const __attribute__((address_space(3))) uint64_t *>(at);
                return static_cast<int>(__builtin_amdgcn_perm(static_cast<uint32_t>(v >> 32), static_cast<uint32_t>(v),
                                                              half ? 0x07060302u : 0x05040100u));
            } else {
                return static_cast<int>(sh.scales[s / kScaleStages & 1][row][2 * half + (s / 2) % 2]);
            }
        };
        auto read_scales = [&](int s, int (&x)[MS], int (&w)[NS]) {
#pragma unroll
            for (int m = 0; m < MS; ++m)
                x[m] = read_scale(s, x0 + 32 * m);
#pragma unroll
            for (int n = 0; n < NS; ++n)
                w[n] = read_scale(s, w0 + 32 * n);
        };
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int m = 0; m < MS; ++m)
                acc[n * kStep][m] = f32x16{};
        // Ungated, the outputs also read sums of columns that only wider wavefronts have, and drop them: any number will do. (Zeros,
        // or a branch at the outputs, cost all tiles more, R131072 E256 H1024 N7168 1033 against 1028 us; gated the branch spares gates,
        // R12288 E128 H4096 N2048 283 -> 278.)
#pragma unroll
        for (int n = NS; n < (GATED ? NS : COLS / 64); ++n)
#pragma unroll
            for (int m = 0; m < MS; ++m)
                asm("" : "=a"(acc[n][m]));
#define MOE_PRODUCTS(STEP, F)                                                                                         \
    _Pragma("unroll") for (int n = 0; n < NS; ++n) _Pragma("unroll") for (int m = 0; m < MS; ++m) acc[n * kStep][m] = \
        __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(F.w[n], F.x[m], acc[n * kStep][m], kFp4, kFp4, STEP, ws[n], STEP, xs[m])
        // the next step's reads, then loads, each before a product of this step
#define MOE_INTERLEAVE(READS, LOADS)                                                                           \
    _Pragma("unroll") for (int i = 0; i < (READS); ++i)                                                        \
    {                                                                                                          \
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                                     \
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                     \
    }                                                                                                          \
    _Pragma("unroll") for (int i = 0; i < (LOADS); ++i)                                                        \
    {                                                                                                          \
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                                                     \
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                     \
    }
        // Every wavefront's loads have come but the LEFT newest of each, and every wavefront has read what it asked for.
        auto meet = [&](auto left) {
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(static_cast<int>(left)) : "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        // Stage s, whose number is J more than an even one: two steps of 64 elements, with the operands of the next step on their
        // way. Between the steps the next stage has come (newer are the loads of two stages), and as every wavefront has read all of
        // this one, loads of the stage kStages on go where it was.
        auto stage = [&](int s, auto J) {
            read(s, 1, f[1]);
#pragma unroll
            for (int j = 0; j < kWLoads; ++j)
                load_w(s + kStages - 1, j);
            MOE_PRODUCTS(2 * J, f[0]);
            MOE_INTERLEAVE(MS + NS, kWLoads);
            meet(std::integral_constant<int, 2 * kLoads>{});
            if constexpr (J == 0 && LINES) {
                const int t = s / 2 + 1;  // the last quarter of a group comes a pair of stages before its first scales are read
                load_line(t / 4 + 1, t % 4);
            } else if constexpr (J == 0) {
                const bool odd = s & 2;
                asm volatile("" : "+v"(sc.x), "+v"(sc.y), "+v"(sc.z), "+v"(sc.w));  // used from here on: before, it would be waited for
                store_sc(!odd, s / kScaleStages + 1);
                load_sc(odd, s / kScaleStages + (odd ? 2 : 1));
            }
            read(s + 1, 0, f[0]);
#pragma unroll
            for (int j = 0; j < kXLoads; ++j)
                load_x(s + kStages, j);
            if constexpr (J == 1)
                read_scales(s + 1, next_xs, next_ws);
            MOE_PRODUCTS(2 * J + 1, f[1]);
            MOE_INTERLEAVE(MS + NS, kXLoads);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (J == 1) {
#pragma unroll
                for (int m = 0; m < MS; ++m)
                    xs[m] = next_xs[m];
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    ws[n] = next_ws[n];
            }
        };
        meet(std::integral_constant<int, 3 * kXLoads + kWLoads>{});  // x's of stages 1 to 3, the weights' of stage 2
        read(0, 0, f[0]);
        read_scales(0, xs, ws);
        for (int s = 0; s < stages; s += 2) {  // after an odd number one of zeros
            stage(s, std::integral_constant<int, 0>{});
            stage(s + 1, std::integral_constant<int, 1>{});
        }
#undef MOE_INTERLEAVE
#undef MOE_PRODUCTS
    };

    // what is left of stages 0 to 2, x's of stage 3, the scales of group 0 and the first of group 1
    const int x_loads = big ? (tile.rows > 192 ? 4 : 3) : tile.rows > 64 ? 2 : 1;
    u32x4 xsc, wsc;
    if constexpr (LINES) {
#pragma unroll
        for (int t = 0; t < 5; ++t)
            load_line(t / 4, t % 4);
    } else {
        if (blocks >= 16) {
            load_sc(false, 0);
            xsc = sc;
            load_sc(true, 0);
            wsc = sc;
        } else {
            xsc = short_scales(xsp, blocks);
            wsc = short_scales(wsp, blocks);
        }
        load_sc(true, 1);
    }
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
#pragma unroll
        for (int j = 0; j < kXMost; ++j)
            if (j < x_loads)
                load_x(s, j);
        if (s == 1)
#pragma unroll
            for (int j = 0; j < kWLoads; ++j)
                load_w(2, j);
    }
    if constexpr (!LINES) {
        put_sc(false, 0, xsc);
        put_sc(true, 0, wsc);
    }
    if constexpr (!kWide)
        tile.rows > 64 ? products(i2, i2, i2) : products(i1, i2, i2);
    else if (tile.rows > 192)
        products(i4, i4, i2);
    else if (big)
        products(i3, i4, i2);
    else if (tile.rows > 64)
        products(i4, i2, i1);
    else if (tile.rows > 32)
        products(i2, i2, i1);
    else
        products(i1, i2, i1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads past the last stage still write zeros
    __syncthreads();

    // Lane l holds row l % 32 of x and, in each four registers, four consecutive weight rows. 32 rows at a time go through LDS, a
    // wavefront's own part of it, and out in vectors of a row.
    constexpr int kMost = (kWide ? 128 : 64) / (GATED ? 2 : 1), kVec = 16 / sizeof(O), kPitch = kMost + kVec, kLanes = kMost / kVec;
    static_assert(4 * 32 * kPitch * sizeof(O) <= sizeof(sh.codes), "");
    // a wavefront's rows and columns
    const int height = !kWide ? (tile.rows > 64 ? 64 : 32) : big && tile.rows <= 192 ? 96 : 128;
    const int row0 = !kWide || big ? wave % 2 * height : 0;
    const int width = GATED ? wave_half : wave_cols;
    const int64_t c0 = n0 + (!kWide || big ? wave / 2 : wave) * width;
    const int cols = static_cast<int>(min(static_cast<int64_t>(width), a.N - c0));
    O *const part = reinterpret_cast<O *>(&sh.codes[0][0]) + wave * 32 * kPitch;
    const bool vectors = a.N % kVec == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
#pragma unroll
    for (int m = 0; m < (kWide ? 4 : 2); ++m) {
        const int rows = min(32, min(height, tile.rows - row0) - 32 * m);
        if (rows <= 0)
            break;
#pragma unroll
        for (int n = 0; n < kMost / 32; ++n) {
            if (GATED && n == kMost / 64 && width < kMost)  // a wavefront of half as many columns has no more sums
                break;
#pragma unroll
            for (int q = 0; q < 16; q += 4) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = GATED ? silu(acc[n][m][q + i]) * acc[n + (GATED ? 2 : 0)][m][q + i] : acc[n][m][q + i];
                put4(part + r32 * kPitch + 32 * n + 2 * q + 4 * half, v);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        O *const out = static_cast<O *>(a.out) + (tile.first + row0 + 32 * m) * a.N + c0;
        if (vectors) {
            const int r0 = lane / kLanes, c = lane % kLanes * kVec;
            O *to = out + r0 * a.N + c;
#pragma unroll
            for (int i = 0; i < 32 * kLanes / kWave; ++i, to += kWave / kLanes * a.N)
                if (r0 + i * (kWave / kLanes) < rows && c < cols)
                    st16(to, ld16(part + (r0 + i * (kWave / kLanes)) * kPitch + c));
        } else {
#pragma unroll 1
            for (int r = 0; r < rows; ++r)
#pragma unroll 1
                for (int c = lane; c < cols; c += kWave)
                    out[r * a.N + c] = part[r * kPitch + c];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// Tiles of BM rows that R rows in E segments can need.
int64_t max_tiles(int64_t R, int64_t E, int64_t BM) { return R / BM + std::min(R, E); }

constexpr int64_t kCus = 256;
constexpr int64_t kMaxGrid = 0xffffffff / kPlanThreads;  // a grid's threads are a 32-bit number

template <typename O, bool GATED>
moe_status launch_product(ProductArgs a, hipStream_t stream)
{
    // Wide tiles, about: with fewer than CUs the tiles of 128 (E8 H4096 N2048, 128 rows an expert 17.6 against 30.4 us; one expert
    // of 2048 rows 19.0 against 31.3; E8 N4096 27.0 against 31.3), otherwise the wide ones (4096 cubed, 256 of them, 44 against 56;
    // R131072 E256 H1024 N7168 1070 against 1271; where experts have few rows and H is short the small ones would win, H1024, 32
    // rows of each of 64: 46 against 41).
    const int64_t experts = std::min(a.R, static_cast<int64_t>(a.E));  // with rows, at most
    const int64_t wide = std::max(experts, a.R / 256) * ceil_div(a.N, GATED ? 128 : 256);
    // Up to 8 rows an expert without tiles (E128 H4096 N2048 gated, 8 rows: 204 against 213 us; E64, 12 rows: 126 against 110), or 16
    // where tiles are few (E8 H4096 N2048, 12 rows: 12.7 against 14.2; 16: 14.3 against 14.2). The host does not know the
    // segments: all rows on one expert, each 16 of which read its weights again, take less than rows on all (2048 rows of E256 H7168
    // N1024 gated 185 against 356). Nor does it know the rows that take part of aligned and drop-and-pad segments, and goes by all: one
    // token of E256 H7168 N1024 gated with segments of multiples of 16 27 us, of 8 20, without alignment 12; 64 tokens 320 and 270.
    const bool few_rows = a.R <= (wide < kCus ? 16 : 8) * static_cast<int64_t>(a.E);
    if (!few_rows) {
        const int size = wide < kCus ? 128 : 256;
        a.col_tiles = static_cast<uint32_t>(ceil_div(a.N, GATED ? size / 2 : size));
        const int64_t tiles = max_tiles(a.R, a.E, size) * a.col_tiles;
        if (tiles > kMaxGrid)
            return MOE_ERR_UNSUPPORTED;
        const dim3 grid(static_cast<unsigned>(tiles));
        const bool far = a.src_row && a.x_rows * (a.H / 2) > kNowhere;
        if (size == 128 && far)
            hipLaunchKernelGGL((grouped_tile_kernel<O, GATED, 128, 128, false, true>), grid, dim3(kPlanThreads), 0, stream, a);
        else if (size == 128)
            hipLaunchKernelGGL((grouped_tile_kernel<O, GATED, 128, 128, false, false>), grid, dim3(kPlanThreads), 0, stream, a);
        else if (far)
            hipLaunchKernelGGL((grouped_tile_kernel<O, GATED, 256, 256, false, true>), grid, dim3(kPlanThreads), 0, stream, a);
        else if (a.H % 512 == 0 && aligned16(a.xs) && aligned16(a.ws))
            hipLaunchKernelGGL((grouped_tile_kernel<O, GATED, 256, 256, true, false>), grid, dim3(kPlanThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((grouped_tile_kernel<O, GATED, 256, 256, false, false>), grid, dim3(kPlanThreads), 0, stream, a);
        return launch_status();
    }
    // Four wavefronts a unit (32 weight rows of an expert's 16 rows) where they all run at once: 512 units of H7168 12.7 against
    // 20.2 us by one, 768 of H4096 12.9 against 15.3, 256 of H1024 4.4 against 5.6; 992 of H4096 18.3 against 14.4, 16384 of H2048
    // 137 against 93. Of H512 there is one run of elements to share.
    const int64_t units = std::max(experts, a.R / 16) * ceil_div(a.N, GATED ? 16 : 32);
    const int split = units <= kRowsWorkgroups * kCus && a.H >= 2 * 2 * kRunBytes ? 4 : 1;
    a.col_tiles = static_cast<uint32_t>(ceil_div(a.N, (GATED ? 16 : 32) * (kPlanThreads / kWave / split)));
    const int64_t tiles = max_tiles(a.R, a.E, 16) * a.col_tiles;
    if (tiles > kMaxGrid)
        return MOE_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(tiles));
    if (split == 4)
        hipLaunchKernelGGL((grouped_rows_kernel<O, GATED, 4>), grid, dim3(kPlanThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((grouped_rows_kernel<O, GATED, 1>), grid, dim3(kPlanThreads), 0, stream, a);
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
