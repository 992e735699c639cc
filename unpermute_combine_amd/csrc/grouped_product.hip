// The products of the experts' rows with their weights, both in microscaled 4-bit floating point:
//   y[r, n] = sum_h X[r, h] W_e[n, h]        for the rows r of expert e's segment, float32 sums
//   out = y, or gated (W_e's first N rows the gate, the next N the up): out[r, n] = silu(y[r, n]) * y[r, N + n]
// A matrix instruction (v_mfma_scale_f32_16x16x128) takes 16 rows of each operand by 128 elements: lane l holds the 32
// elements of block l / 16 of row l % 16, and the block's scale.
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
// cubed 334 -> 298 us against all the rows' tiles first.)
constexpr uint32_t kGroup = 8;
// Every thread of a workgroup of kPlanThreads calls it and gets the same.
template <int BM>
__device__ __forceinline__ Tile find_tile(const ProductArgs &a, uint32_t i)
{
    __shared__ uint32_t wave_tiles[kPlanThreads / kWave];
    __shared__ Tile found;
    constexpr int kPer = MOE_MAX_EXPERTS / kPlanThreads;
    const int per = static_cast<int>((a.E + kPlanThreads - 1) / kPlanThreads), e0 = threadIdx.x * per;
    uint32_t tiles[kPer], start[kPer], len[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        tiles[j] = start[j] = len[j] = 0;
        if (j < per && e0 + j < a.E) {
            int64_t s, l;
            segment(a, e0 + j, s, l);
            start[j] = static_cast<uint32_t>(s);
            len[j] = static_cast<uint32_t>(l);
            tiles[j] = (len[j] + BM - 1) / BM * a.col_tiles;
            mine += tiles[j];
        }
    }
    // (the launch has made sure that their number fits)
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    uint32_t upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t o = __shfl_up(upto, d);
        upto += lane >= d ? o : 0;
    }
    if (lane == kWave - 1)
        wave_tiles[wave] = upto;
    if (threadIdx.x == 0)
        found = Tile{-1, 0, 0, 0};
    __syncthreads();
    uint32_t k = i - (upto - mine);
#pragma unroll
    for (int v = 0; v < kPlanThreads / kWave - 1; ++v)
        k -= v < wave ? wave_tiles[v] : 0;
    if (k < mine) {  // (before this thread's tiles k is negative, as a large number)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (k < tiles[j]) {
                const uint32_t n = (len[j] + BM - 1) / BM, g = k / (kGroup * a.col_tiles), in = k % (kGroup * a.col_tiles);
                const uint32_t high = min(kGroup, n - kGroup * g), m = kGroup * g + in % high;
                found = Tile{e0 + j, static_cast<int32_t>(min(len[j] - m * BM, static_cast<uint32_t>(BM))),
                             static_cast<int64_t>(start[j]) + m * BM, static_cast<int32_t>(in / high)};
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
__device__ __forceinline__ float silu(float g)
{
    constexpr float kLog2e = 1.44269504088896340736f;
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * g));
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

// A wavefront's share of 512 elements: 32 weight rows, 16 rows of x, and their scales.
struct Run {
    u32x4 w[2][4], x[4], ws[2], xs;
};

// Up to 16 rows of an expert by 32 weight rows (gated: 16 of the gate and the 16 of the up of the same columns) a wavefront. The
// weights go from memory into the matrix instructions' operand registers, the next 512 elements on their way while these are
// multiplied. SPLIT wavefronts share the columns and take parts of the sum, put together in LDS.
template <typename O, bool GATED, int SPLIT>
__global__ __launch_bounds__(kPlanThreads) void grouped_rows_kernel(ProductArgs a)
{
    constexpr int kWaves = kPlanThreads / kWave, kCols = GATED ? 16 : 32;  // columns a wavefront
    __shared__ f32x4 sums[SPLIT > 1 ? kWaves : 1][2][kWave];
    const Tile tile = find_tile<16>(a, blockIdx.x);
    if (tile.e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / kWave));
    const int r = lane & 15, g = lane >> 4, part = wave % SPLIT;
    const int64_t n0 = (static_cast<int64_t>(tile.col) * (kWaves / SPLIT) + wave / SPLIT) * kCols;
    const int blocks = static_cast<int>(a.H / kMxBlock), runs = (blocks + kRunBlocks - 1) / kRunBlocks;
    const int64_t row_bytes = a.H / 2, wrows = a.N * (GATED ? 2 : 1);
    f32x4 acc[2] = {};
    if (n0 < a.N) {
        // x's row r, and the scales' row r of each 16 weight rows
        int64_t row = tile.first + min(r, tile.rows - 1);
        bool there = r < tile.rows;
        if (a.src_row) {
            row = a.src_row[row];
            there = there && row >= 0 && row < a.x_rows;
            row = there ? row : 0;
        }
        const uint8_t *const x = a.x + row * row_bytes, *const xs = there ? a.xs + row * blocks : a.ws;
        // the weight rows from w_at(i) on; of the last columns' those past the end are the last one
        auto w_at = [&](int i) { return tile.e * wrows + n0 + (GATED ? i * a.N : 16 * i); };
        auto last = [&](int i) { return static_cast<int>(min(a.N - n0 - (GATED ? 0 : 16 * i), int64_t{16})) - 1; };
        uint32_t wo[2][2];
        const uint8_t *ws[2];
        __amdgpu_buffer_rsrc_t wr[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int end = max(last(i), 0);
            const int64_t at = min(w_at(i), a.E * wrows - 1);
            wr[i] = make_rsrc(a.w + at * row_bytes, static_cast<uint32_t>(min((a.E * wrows - at) * row_bytes, int64_t{0xfffffff0})));
#pragma unroll
            for (int j = 0; j < 2; ++j)
                wo[i][j] = static_cast<uint32_t>(min(8 * j + (r & 7), end) * row_bytes) + (g + (r & 8) / 2) * 16;
            ws[i] = a.ws + (at + min(r, end)) * blocks;
        }
        auto scales = [&](const uint8_t *from, int run) -> u32x4 {
            if (blocks < kRunBlocks)
                return short_scales(from, blocks);
            u32x4 v;
            __builtin_memcpy(&v, from + min(run * kRunBlocks, blocks - kRunBlocks), sizeof(v));
            return v;
        };
        auto load = [&](int run, Run &to) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    to.w[i][j] = ld16_buf<0>(wr[i], wo[i][j & 1] + run * kRunBytes + (j >> 1) * 128);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int b = run * kRunBlocks + 4 * j + g;
                to.x[j] = u32x4{0, 0, 0, 0};
                if (there && b < blocks)
                    to.x[j] = ld16(x + b * 16);
            }
            to.ws[0] = scales(ws[0], run);
            to.ws[1] = scales(ws[1], run);
            to.xs = scales(xs, run);
        };
        auto multiply = [&](int run, Run &f) {
            const int past = blocks < kRunBlocks ? 0 : run * kRunBlocks - min(run * kRunBlocks, blocks - kRunBlocks);
            const u32x4 sx = shifted(f.xs, past);
            const uint32_t keep = there ? 0xffffffffu : 0;
            const uint32_t s[4] = {sx.x & keep, sx.y & keep, sx.z & keep, sx.w & keep};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x4 sw = shifted(f.ws[i], past);
                const uint32_t t[4] = {sw.x, sw.y, sw.z, sw.w};
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    u32x4 &p = f.w[i][j], &q = f.w[i][j + 1];
                    swap_eights(p.x, q.x);
                    swap_eights(p.y, q.y);
                    swap_eights(p.z, q.z);
                    swap_eights(p.w, q.w);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        operand(f.w[i][j]), operand(f.x[j]), acc[i], kFp4, kFp4, 0, static_cast<int>(t[j] >> (8 * g)), 0,
                        static_cast<int>(s[j] >> (8 * g)));
            }
        };
        const int from = runs * part / SPLIT, to = runs * (part + 1) / SPLIT;
        if (from < to) {
            Run f[2];
            load(from, f[0]);
            int run = from;
            for (; run + 2 < to; run += 2) {
                load(run + 1, f[1]);
                multiply(run, f[0]);
                load(run + 2, f[0]);
                multiply(run + 1, f[1]);
            }
            if (run + 1 < to) {
                load(run + 1, f[1]);
                multiply(run, f[0]);
                multiply(run + 1, f[1]);
            } else {
                multiply(run, f[0]);
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
    // lane l holds row l % 16 and four consecutive columns of each 16
    if (r >= tile.rows)
        return;
    O *const out = static_cast<O *>(a.out) + (tile.first + r) * a.N;
    const bool vectors = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & (4 * sizeof(O) - 1)) == 0;
#pragma unroll
    for (int i = 0; i < (GATED ? 1 : 2); ++i) {
        const int64_t c = n0 + 16 * i + 4 * g;
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = GATED ? silu(acc[0][q]) * acc[1][q] : acc[i][q];
        if (vectors) {
            if (c < a.N)
                put4(out + c, v);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (c + q < a.N)
                    store_out(out + c + q, v[q]);
        }
    }
}

// ---------------------------------------------------------------- tiles through LDS

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileRows = 256, kTileCols = 256;  // rows and weight rows of the largest tile
constexpr int kStageBytes = 64;                  // of each row a stage: 128 elements
constexpr int kStageBlocks = kStageBytes / 16;
constexpr int kStages = 4;                       // of which LDS has room
constexpr int kScaleStages = 4;                  // stages whose scales come at a time: 16 bytes of a row

// The 16-byte chunk c of row r lies in slot c ^ swizzle(r) of its 64 bytes: 8 and 16 consecutive rows' same chunk fall into
// different banks.
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); }

struct Buffers {
    uint8_t codes[kStages][(kTileRows + kTileCols) * kStageBytes];
    uint32_t scales[2][kTileRows + kTileCols][4];
};

// 16 bytes a lane into LDS, lane l's to address `to` + 16 l (one for the wavefront). Past the resource's end: zeros.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, uint32_t to)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, reinterpret_cast<__attribute__((address_space(3))) void *>(to), 16,
                                             static_cast<int>(offset), 0, 0, 0);
}

__device__ __forceinline__ uint32_t capped(int64_t bytes)
{
    return static_cast<uint32_t>(min(bytes, static_cast<int64_t>(0xffffffffu)));
}

template <int MS, int NS>
struct Frags {
    i32x8 x[MS], w[NS];
};

// A tile of up to 32 MS WM rows by 256 weight rows (gated: 128 of the gate and 128 of the up), four wavefronts, WM beside each
// other along the rows: a wavefront has 32 MS rows by 32 NS weight rows.
template <typename O, bool GATED, int MS, int NS, int WM>
__device__ __forceinline__ void tile_product(const ProductArgs &a, const Tile &tile, Buffers &sh)
{
    constexpr int kRows = 32 * MS * WM, kWN = 4 / WM;  // wavefronts along the columns
    static_assert(32 * NS * kWN == kTileCols, "");
    constexpr int kWaveCols = 32 * NS, kHalf = kWaveCols / 2;
    constexpr int kOutCols = GATED ? kTileCols / 2 : kTileCols;
    constexpr int kXLoads = kRows < 64 ? 1 : kRows / 64, kWLoads = kTileCols / 64;  // 16-byte loads a thread and stage
    constexpr int kLoads = kXLoads + kWLoads, kEarly = kLoads / 2;
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / kWave));
    const int blocks = static_cast<int>(a.H / kMxBlock), stages = (blocks + kStageBlocks - 1) / kStageBlocks;
    const int64_t row_bytes = a.H / 2, n0 = static_cast<int64_t>(tile.col) * kOutCols;

    // the row of x behind row r of the tile (any one where there is none: the epilogue drops it)
    auto x_row = [&](int r) -> int64_t {
        int64_t row = tile.first + min(r, tile.rows - 1);
        if (a.src_row) {
            row = a.src_row[row];
            row = row >= 0 && row < a.x_rows ? row : 0;
        }
        return row;
    };
    // the weight row, from n0 on, behind row b of the tile's weights: gated, a wavefront's first half are gates, its second the ups
    // of the same columns (is_up)
    auto w_row = [&](int b) -> int64_t {
        const int64_t n = GATED ? b / kWaveCols * kHalf + b % kHalf : b;
        return min(n, a.N - 1 - n0);
    };
    auto is_up = [&](int b) { return GATED && b % kWaveCols >= kHalf; };

    // A load takes 16 rows a wavefront, 4 lanes a row: thread t chunk slot t % 4 of rows 64 j + t / 4. Loads go by buffer resources,
    // whose bounds keep what lies past the last row's end unread. x is from its tile's first row on, or whole with a map.
    const int chunk = (lane & 3) ^ swizzle(lane >> 2);
    const int64_t x_at = a.src_row ? 0 : tile.first;
    const uint8_t *xbase = a.x + x_at * row_bytes;
    const uint32_t xbytes = capped((a.x_rows - x_at) * row_bytes);
    const int64_t wrows = a.N * (GATED ? 2 : 1), w_at = tile.e * wrows + n0;
    uint32_t xo[kXLoads], wo[kWLoads];
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
        xo[j] = static_cast<uint32_t>((x_row(64 * j + threadIdx.x / 4) - x_at) * row_bytes) + chunk * 16;
#pragma unroll
    for (int j = 0; j < kWLoads; ++j)
        wo[j] = static_cast<uint32_t>(w_row(64 * j + threadIdx.x / 4) * row_bytes) + chunk * 16;
    const uint8_t *xsp = a.x_rows > 0 ? a.xs + x_row(threadIdx.x) * blocks : a.ws;  // (any, where x has no rows)
    const uint8_t *wsp = a.ws + (w_at + w_row(threadIdx.x) + (is_up(threadIdx.x) ? a.N : 0)) * blocks;

    // The stages' addresses as plain numbers: of what it sees to lie in the array the compiler would wait for every load under
    // way into it, those of later stages included, before each read. What a read needs has come by `meet`.
    uint32_t codes = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)&sh.codes[0][0]));
    asm volatile("" : "+s"(codes));
    // Loads FROM to TO of stage s. x's chunks past the end of the rows are zeros (beside them the weights' are some codes, and zero
    // times them is zero); past the last stage nothing is read, but the number of loads is the same in every stage.
    auto issue = [&](int s, auto from, auto to) {
        const uint32_t at = codes + (s % kStages) * sizeof(sh.codes[0]) + wave * 16 * kStageBytes, k = s * kStageBytes;
        const bool there = s < stages, in_row = s * kStageBlocks + chunk < blocks;
#pragma unroll
        for (int j = from; j < to; ++j) {
            if (j < kXLoads) {
                to_lds(make_rsrc(xbase, xbytes), in_row ? xo[j] + k : 0xfffffff0u, at + 64 * j * kStageBytes);
            } else {
                const int i = j - kXLoads;
                const int64_t row = w_at + (is_up(64 * i + 16 * wave) ? a.N : 0);
                to_lds(make_rsrc(a.w + row * row_bytes, there ? capped((a.E * wrows - row) * row_bytes) : 0), wo[i] + k,
                       at + (kTileRows + 64 * i) * kStageBytes);
            }
        }
    };
    const auto none = std::integral_constant<int, 0>{};
    const auto early = std::integral_constant<int, kEarly>{};
    const auto all = std::integral_constant<int, kLoads>{};

    // Scales come for kScaleStages stages (a group) at a time, x's and the weights' in turns: thread t has row t's. A row's 16 bytes
    // are put down as what each half of a wavefront needs of them: blocks 0, 1 of each stage's four, then blocks 2, 3.
    const uint8_t *const xsl = blocks >= 16 ? xsp : a.w, *const wsl = blocks >= 16 ? wsp : a.w;  // (rows of 16 bytes to read)
    u32x4 sc;
    auto load_sc = [&](bool w, int g) {  // past the end: what nothing uses
        __builtin_memcpy(&sc, (w ? wsl : xsl) + max(min(16 * g, blocks - 16), 0), sizeof(sc));
    };
    auto put_sc = [&](bool w, int g, const u32x4 &v) {
        st16(sh.scales[g & 1][(w ? kTileRows : 0) + threadIdx.x],
             u32x4{__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                   __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)});
    };
    auto store_sc = [&](bool w, int g) { put_sc(w, g, shifted(sc, min(16 * g - max(min(16 * g, blocks - 16), 0), 15))); };

    const int half = lane >> 5, r32 = lane & 31;
    const int x0 = (wave % WM) * 32 * MS + r32, w0 = kTileRows + (wave / WM) * kWaveCols + r32;
    // a lane's 16 bytes in steps 0 and 1 of a stage: chunks 2 half and 2 half + 1
    const uint32_t lane_at[2] = {codes + x0 * kStageBytes + ((2 * half) ^ swizzle(r32)) * 16,
                                 codes + x0 * kStageBytes + ((2 * half + 1) ^ swizzle(r32)) * 16};
    auto frag = [&](int s, int row, int ks) -> i32x8 {
        const uint32_t at = lane_at[ks] + (s % kStages) * sizeof(sh.codes[0]) + row * kStageBytes;
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
    auto read_scales = [&](int s, int (&x)[MS], int (&w)[NS]) {
        const int word = 2 * half + (s / 2) % 2, g = s / kScaleStages & 1;
#pragma unroll
        for (int m = 0; m < MS; ++m)
            x[m] = static_cast<int>(sh.scales[g][x0 + 32 * m][word]);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            w[n] = static_cast<int>(sh.scales[g][w0 + 32 * n][word]);
    };

    f32x16 acc[NS][MS];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int m = 0; m < MS; ++m)
            acc[n][m] = f32x16{};
#define MOE_PRODUCTS(STEP, F)                                                                                         \
    _Pragma("unroll") for (int n = 0; n < NS; ++n) _Pragma("unroll") for (int m = 0; m < MS; ++m) acc[n][m] =         \
        __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(F.w[n], F.x[m], acc[n][m], kFp4, kFp4, STEP, ws[n], STEP, xs[m])
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
    // Stage s, whose number is J more than an even one: two steps of 64 elements, with the operands of the next step on their way.
    // Between the steps the next stage has come, and as every wavefront has read all of this one, loads of the stage kStages on go
    // where it was.
    auto stage = [&](int s, auto J) {
        read(s, 1, f[1]);
        issue(s + kStages - 1, early, all);
        MOE_PRODUCTS(2 * J, f[0]);
        MOE_INTERLEAVE(MS + NS, kLoads - kEarly);
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (J == 0) {
            const bool odd = s & 2;
            asm volatile("" : "+v"(sc.x), "+v"(sc.y), "+v"(sc.z), "+v"(sc.w));  // used from here on: before, it would be waited for
            store_sc(!odd, s / kScaleStages + 1);
            load_sc(odd, s / kScaleStages + (odd ? 2 : 1));
        }
        read(s + 1, 0, f[0]);
        issue(s + kStages, none, early);
        if constexpr (J == 1)
            read_scales(s + 1, next_xs, next_ws);
        MOE_PRODUCTS(2 * J + 1, f[1]);
        MOE_INTERLEAVE(MS + NS, kEarly);
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
    issue(0, none, all);
    if (blocks >= 16) {
        load_sc(false, 0);
        const u32x4 x = sc;
        load_sc(true, 0);
        const u32x4 w = sc;
        load_sc(true, 1);
#pragma unroll
        for (int s = 1; s < kStages - 1; ++s)
            issue(s, none, all);
        issue(kStages - 1, none, early);
        put_sc(false, 0, x);
        put_sc(true, 0, w);
    } else {
        load_sc(true, 1);
#pragma unroll
        for (int s = 1; s < kStages - 1; ++s)
            issue(s, none, all);
        issue(kStages - 1, none, early);
        put_sc(false, 0, short_scales(xsp, blocks));
        put_sc(true, 0, short_scales(wsp, blocks));
    }
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * kLoads + kEarly) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(0, 0, f[0]);
    read_scales(0, xs, ws);
    for (int s = 0; s < stages; s += 2) {  // after an odd number one of zeros
        stage(s, std::integral_constant<int, 0>{});
        stage(s + 1, std::integral_constant<int, 1>{});
    }
#undef MOE_INTERLEAVE
#undef MOE_PRODUCTS
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads past the last stage still write zeros
    // Lane l holds row l % 32 of x and, in each four registers, four consecutive weight rows. 32 rows at a time go through LDS, a
    // wavefront's own part of it, and out in whole vectors of a row.
    constexpr int kOut = GATED ? kHalf : kWaveCols, kPad = 16 / sizeof(O), kPitch = kOut + kPad, kVec = 16 / sizeof(O);
    static_assert(4 * 32 * kPitch * sizeof(O) <= sizeof(sh.codes), "");
    __syncthreads();
    O *part = reinterpret_cast<O *>(&sh.codes[0][0]) + wave * 32 * kPitch;
    const int64_t c0 = n0 + (wave / WM) * kOut;
    const int cols = static_cast<int>(min(static_cast<int64_t>(kOut), a.N - c0));
    const bool vectors = a.N % kVec == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        const int r0 = (wave % WM) * 32 * MS + 32 * m, rows = min(32, tile.rows - r0);
        if (rows <= 0)
            break;
        bool there = true;
        if (a.src_row && r32 < rows) {
            const int64_t from = a.src_row[tile.first + r0 + r32];
            there = from >= 0 && from < a.x_rows;
        }
#pragma unroll
        for (int n = 0; n < (GATED ? NS / 2 : NS); ++n)
#pragma unroll
            for (int q = 0; q < 16; q += 4) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = GATED ? silu(acc[n][m][q + i]) * acc[n + NS / 2][m][q + i] : acc[n][m][q + i];
                    v[i] = there ? v[i] : 0.0f;
                }
                put4(part + r32 * kPitch + 32 * n + 2 * q + 4 * half, v);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        O *out = static_cast<O *>(a.out) + (tile.first + r0) * a.N + c0;
        if (vectors) {
            constexpr int kLanes = kOut / kVec;  // lanes a row
#pragma unroll
            for (int i = 0; i < 32 * kLanes / kWave; ++i) {
                const int r = i * (kWave / kLanes) + lane / kLanes, c = lane % kLanes * kVec;
                if (r < rows && c < cols)
                    st16(out + r * a.N + c, ld16(part + r * kPitch + c));
            }
        } else {
            for (int r = 0; r < rows; ++r)
                for (int c = lane; c < cols; c += kWave)
                    out[r * a.N + c] = part[r * kPitch + c];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// Workgroup b of nb, dealt to the XCDs in turn, takes the place that keeps runs of kRun neighbours on one XCD.
constexpr uint32_t kRun = 16;
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t nb)
{
    const uint32_t round = b / (kXcds * kRun), in = b % (kXcds * kRun);
    return (round + 1) * kXcds * kRun > nb ? b : round * kXcds * kRun + in % kXcds * kRun + in / kXcds;
}

template <typename O, bool GATED>
__global__ __launch_bounds__(kPlanThreads) void grouped_tile_kernel(ProductArgs a)
{
    __shared__ __attribute__((aligned(128))) Buffers sh;
    const Tile tile = find_tile<kTileRows>(a, xcd_run(blockIdx.x, gridDim.x));
    if (tile.e < 0)
        return;
    if (tile.rows > 128)
        tile_product<O, GATED, 4, 4, 2>(a, tile, sh);
    else if (tile.rows > 64)
        tile_product<O, GATED, 4, 2, 1>(a, tile, sh);
    else if (tile.rows > 32)
        tile_product<O, GATED, 2, 2, 1>(a, tile, sh);
    else
        tile_product<O, GATED, 1, 2, 1>(a, tile, sh);
}

// Tiles of BM rows that R rows in E segments can need.
int64_t max_tiles(int64_t R, int64_t E, int64_t BM) { return R / BM + std::min(R, E); }

constexpr int64_t kFewUnits = 4096;

template <typename O, bool GATED>
moe_status launch_product(ProductArgs a, hipStream_t stream)
{
    // (rows through a map are addressed in 32 bits there)
    if (a.R > 16 * static_cast<int64_t>(a.E) && (!a.src_row || a.x_rows * (a.H / 2) <= 0xffffffff)) {
        a.col_tiles = static_cast<uint32_t>(ceil_div(a.N, GATED ? kTileCols / 2 : kTileCols));
        const int64_t grid = max_tiles(a.R, a.E, kTileRows) * a.col_tiles;
        if (grid > 0x7fffffff)
            return MOE_ERR_UNSUPPORTED;
        hipLaunchKernelGGL((grouped_tile_kernel<O, GATED>), dim3(static_cast<unsigned>(grid)), dim3(kPlanThreads), 0, stream, a);
        return launch_status();
    }
    const int64_t tiles = max_tiles(a.R, a.E, 16), units = tiles * ceil_div(a.N, GATED ? 16 : 32);
    const int split = units < kFewUnits && a.H >= 4 * 512 ? 4 : 1;
    a.col_tiles = static_cast<uint32_t>(ceil_div(a.N, (GATED ? 16 : 32) * (kPlanThreads / kWave / split)));
    if (tiles * a.col_tiles > 0x7fffffff)
        return MOE_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(tiles * a.col_tiles));
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
