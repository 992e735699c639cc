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

// The i-th of the (rows, columns) tiles of BM rows, experts in order, an expert's tiles of the same columns beside each other.
// Every thread of a workgroup of kPlanThreads calls it and gets the same.
template <int BM>
__device__ __forceinline__ Tile find_tile(const ProductArgs &a, int64_t i)
{
    __shared__ int64_t wave_tiles[kPlanThreads / kWave];
    __shared__ Tile found;
    constexpr int kPer = MOE_MAX_EXPERTS / kPlanThreads;
    const int per = static_cast<int>(ceil_div(a.E, kPlanThreads));
    const int e0 = threadIdx.x * per;
    int64_t tiles[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        tiles[j] = 0;
        if (j < per && e0 + j < a.E) {
            int64_t start, len;
            segment(a, e0 + j, start, len);
            tiles[j] = ceil_div(len, BM);
            mine += tiles[j];
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
        found = Tile{-1, 0, 0, 0};
    __syncthreads();
    int64_t before = upto - mine;
    for (int v = 0; v < wave; ++v)
        before += wave_tiles[v];
    int64_t k = i - before * a.col_tiles;
    if (k >= 0 && k < mine * a.col_tiles) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (k >= 0 && k < tiles[j] * a.col_tiles) {
                int64_t start, len;
                segment(a, e0 + j, start, len);
                const int64_t m = k % tiles[j];
                found = Tile{e0 + j, static_cast<int32_t>(min(len - m * BM, int64_t{BM})), start + m * BM,
                             static_cast<int32_t>(k / tiles[j])};
            }
            k -= tiles[j] * a.col_tiles;
        }
    }
    __syncthreads();
    return found;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

__device__ __forceinline__ void store_out(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_out(uint16_t *p, float v) { *p = static_cast<uint16_t>(f32_to_bf16_bits(v)); }

// Four values into LDS.
__device__ __forceinline__ void put4(float *p, const float (&v)[4]) { *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ void put4(uint16_t *p, const float (&v)[4])
{
    *reinterpret_cast<uint64_t *>(p) = pack_bf16x2(v[0], v[1]) | static_cast<uint64_t>(pack_bf16x2(v[2], v[3])) << 32;
}

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
    const Tile tile = find_tile<16>(a, blockIdx.x);
    if (tile.e < 0)
        return;
    const int lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
    const int64_t n0 = (static_cast<int64_t>(tile.col) * (kPlanThreads / kWave) + threadIdx.x / kWave) * 16;
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

// ---------------------------------------------------------------- tiles through LDS

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTileRows = 256, kTileCols = 256;  // rows and weight rows of the largest tile
constexpr int kStageBytes = 128;                 // of each row a stage: 256 elements, a cache line
constexpr int kStageBlocks = kStageBytes / 16;

// The 16-byte chunk c of row r lies in slot c ^ swizzle(r) of its 128 bytes: 8 and 16 consecutive rows' same chunk fall into
// different banks.
__device__ __forceinline__ int swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }

struct Buffers {
    uint8_t codes[2][(kTileRows + kTileCols) * kStageBytes];
    uint64_t scales[2][kTileRows + kTileCols];
};

// Scale bytes of 8 blocks of a row from block b on, the last 8 of the row where fewer are left (rows of 8 blocks at least).
__device__ __forceinline__ uint64_t load_scales(const uint8_t *row, int b, int blocks)
{
    uint64_t v;
    __builtin_memcpy(&v, row + min(b, blocks - 8), 8);
    return v;
}

// Of what load_scales gave, the bytes from block b on in their places; past the row's end any but NaN.
__device__ __forceinline__ uint64_t placed_scales(uint64_t v, int b, int blocks)
{
    return v >> (8 * (b - min(b, blocks - 8)));
}

// The scale bytes of a row of fewer than 8 blocks.
__device__ __forceinline__ uint64_t short_scales(const uint8_t *row, int blocks)
{
    uint64_t v = 0;
    for (int i = 0; i < blocks; ++i)
        v |= static_cast<uint64_t>(row[i]) << (8 * i);
    return v;
}

// 16 bytes a lane into LDS, lane l's to address `to` + 16 l (one for the wavefront).
__device__ __forceinline__ void to_lds(const uint8_t *from, uint32_t to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     reinterpret_cast<__attribute__((address_space(3))) void *>(to), 16, 0, 0);
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
    constexpr int kXLoads = kRows / 32, kWLoads = kTileCols / 32;  // 16-byte loads a thread and stage
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / kWave));
    const int blocks = static_cast<int>(a.H / kMxBlock), stages = (blocks + kStageBlocks - 1) / kStageBlocks;
    const int64_t row_bytes = a.H / 2, n0 = static_cast<int64_t>(tile.col) * kOutCols;
    const uint8_t *xbase = a.x_rows > 0 ? a.x : a.w, *xsbase = a.x_rows > 0 ? a.xs : a.ws;

    // the row of x behind row r of the tile (any one where there is none: the epilogue drops it)
    auto x_row = [&](int r) -> int64_t {
        int64_t row = tile.first + min(r, tile.rows - 1);
        if (a.src_row) {
            row = a.src_row[row];
            row = row >= 0 && row < a.x_rows ? row : 0;
        }
        return row;
    };
    // the weight row behind row b of the tile's weights: gated, a wavefront's first half are gates and its second the ups of them
    auto w_row = [&](int b) -> int64_t {
        if (!GATED)
            return tile.e * a.N + min(n0 + b, a.N - 1);
        const int in = b % kWaveCols;
        const int64_t n = min(n0 + b / kWaveCols * kHalf + in % kHalf, a.N - 1);
        return tile.e * 2 * a.N + n + (in >= kHalf ? a.N : 0);
    };

    // thread t loads chunk slot t % 8 of rows t / 8 + 32 j
    const int chunk = (lane & 7) ^ swizzle(threadIdx.x / 8);
    const uint8_t *xp[kXLoads], *wp[kWLoads];
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
        xp[j] = xbase + x_row(threadIdx.x / 8 + 32 * j) * row_bytes;
#pragma unroll
    for (int j = 0; j < kWLoads; ++j)
        wp[j] = a.w + w_row(threadIdx.x / 8 + 32 * j) * row_bytes;
    const uint8_t *xsp = xsbase + x_row(min(static_cast<int>(threadIdx.x), kRows - 1)) * blocks;
    const uint8_t *wsp = a.ws + w_row(threadIdx.x) * blocks;

    // The stages' addresses as plain numbers: of what it sees to lie in the array the compiler would wait for every load under
    // way into it, those of the next stage included, before each read. What a read needs has come by `meet`.
    uint32_t codes = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)&sh.codes[0][0]));
    asm volatile("" : "+s"(codes));
    auto issue = [&](int s) {
        const uint32_t to = codes + (s & 1) * sizeof(sh.codes[0]) + wave * 8 * kStageBytes;
        const int at = min(s * kStageBlocks + chunk, blocks - 1) * 16;  // past the end: any chunk
#pragma unroll
        for (int j = 0; j < kXLoads; ++j)
            to_lds(xp[j] + at, to + 32 * j * kStageBytes);
#pragma unroll
        for (int j = 0; j < kWLoads; ++j)
            to_lds(wp[j] + at, to + (kTileRows + 32 * j) * kStageBytes);
    };
    uint64_t xsc, wsc;
    auto load_sc = [&](int s) {  // (past the last stage: what nothing uses)
        xsc = load_scales(xsp, s * kStageBlocks, blocks);
        wsc = load_scales(wsp, s * kStageBlocks, blocks);
    };
    auto store_sc = [&](int s) {
        sh.scales[s & 1][threadIdx.x] = placed_scales(xsc, s * kStageBlocks, blocks);
        sh.scales[s & 1][kTileRows + threadIdx.x] = placed_scales(wsc, s * kStageBlocks, blocks);
    };
    // chunks past the end of the rows: zeros for x (the weights' are some codes, and zero times them is zero)
    auto clear_tail = [&]() {
        if (blocks % kStageBlocks == 0)
            return;
        uint8_t *x = sh.codes[(stages - 1) & 1];
        for (int i = threadIdx.x; i < kRows * kStageBlocks; i += kPlanThreads) {
            const int r = i / kStageBlocks, c = i % kStageBlocks;
            if (c >= blocks % kStageBlocks)
                *reinterpret_cast<i32x4 *>(x + r * kStageBytes + (c ^ swizzle(r)) * 16) = i32x4{0, 0, 0, 0};
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    const int half = lane >> 5, r32 = lane & 31;
    const int x0 = (wave % WM) * 32 * MS + r32, w0 = kTileRows + (wave / WM) * kWaveCols + r32;
    const int swz = swizzle(r32);
    auto frag = [&](int s, int row, int ks) -> i32x8 {
        const uint32_t at = codes + (s & 1) * sizeof(sh.codes[0]) + row * kStageBytes + ((4 * half + ks) ^ swz) * 16;
        const i32x4 v = *reinterpret_cast<const __attribute__((address_space(3))) i32x4 *>(at);
        return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
    };
    auto scale = [&](int s, int row) -> int {
        return reinterpret_cast<const int *>(sh.scales[s & 1] + row)[half];
    };

    f32x16 acc[NS][MS];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int m = 0; m < MS; ++m)
            acc[n][m] = f32x16{};
    Frags<MS, NS> f[2];
    int xs[2][MS], ws[2][NS];
    auto read = [&](int s, int ks, Frags<MS, NS> &to) {
#pragma unroll
        for (int m = 0; m < MS; ++m)
            to.x[m] = frag(s, x0 + 32 * m, ks);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            to.w[n] = frag(s, w0 + 32 * n, ks);
    };
    auto read_scales = [&](int s, int (&x)[MS], int (&w)[NS]) {
#pragma unroll
        for (int m = 0; m < MS; ++m)
            x[m] = scale(s, x0 + 32 * m);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            w[n] = scale(s, w0 + 32 * n);
    };
    auto meet = [&]() {  // what each wavefront asked for has come, and what it read has been read
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
#define MOE_PRODUCTS(KS, F)                                                                                           \
    _Pragma("unroll") for (int n = 0; n < NS; ++n) _Pragma("unroll") for (int m = 0; m < MS; ++m) acc[n][m] =         \
        __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(F.w[n], F.x[m], acc[n][m], kFp4, kFp4, KS, ws[0][n], KS, xs[0][m])
    // the reads of the next step go between the first products of this one
#define MOE_INTERLEAVE()                                                   \
    _Pragma("unroll") for (int i = 0; i < MS + NS; ++i)                    \
    {                                                                      \
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                 \
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                 \
    }                                                                      \
    __builtin_amdgcn_sched_group_barrier(0x008, MS *NS, 0)
    // A stage: four steps of 64 elements, the operands of the next step on their way. Before the last step the next stage has come
    // (turn), and as every wavefront has read all of this one the loads of the stage after it go where this one was (more).
    auto stage = [&](int s, auto turn, auto more) {
        read(s, 1, f[1]);
        MOE_PRODUCTS(0, f[0]);
        MOE_INTERLEAVE();
        read(s, 2, f[0]);
        MOE_PRODUCTS(1, f[1]);
        MOE_INTERLEAVE();
        read(s, 3, f[1]);
        MOE_PRODUCTS(2, f[0]);
        MOE_INTERLEAVE();
        if constexpr (turn) {
            meet();
            if constexpr (!more)
                clear_tail();
            read(s + 1, 0, f[0]);
            read_scales(s + 1, xs[1], ws[1]);
            if constexpr (more) {
                asm volatile("" : "+v"(xsc), "+v"(wsc));  // used from here on: before, they would be waited for
                issue(s + 2);
                store_sc(s + 2);
                load_sc(s + 3);
            }
        }
        MOE_PRODUCTS(3, f[1]);
        if constexpr (turn) {
#pragma unroll
            for (int m = 0; m < MS; ++m)
                xs[0][m] = xs[1][m];
#pragma unroll
            for (int n = 0; n < NS; ++n)
                ws[0][n] = ws[1][n];
        }
    };
    issue(0);
    if (blocks >= 8) {
        load_sc(0);
        store_sc(0);
    } else {
        sh.scales[0][threadIdx.x] = short_scales(xsp, blocks);
        sh.scales[0][kTileRows + threadIdx.x] = short_scales(wsp, blocks);
    }
    if (stages > 1) {
        issue(1);
        load_sc(1);
        store_sc(1);
        load_sc(2);
    }
    meet();
    if (stages == 1)
        clear_tail();
    read(0, 0, f[0]);
    read_scales(0, xs[0], ws[0]);
    int s = 0;
    for (; s < stages - 2; ++s)
        stage(s, std::true_type{}, std::true_type{});
    if (s < stages - 1)
        stage(s++, std::true_type{}, std::false_type{});
    stage(s, std::false_type{}, std::false_type{});
#undef MOE_PRODUCTS
#undef MOE_INTERLEAVE
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

template <typename O, bool GATED>
moe_status launch_product(ProductArgs a, hipStream_t stream)
{
    if (a.R > 16 * static_cast<int64_t>(a.E)) {
        a.col_tiles = static_cast<uint32_t>(ceil_div(a.N, GATED ? kTileCols / 2 : kTileCols));
        const int64_t grid = max_tiles(a.R, a.E, kTileRows) * a.col_tiles;
        if (grid > 0x7fffffff)
            return MOE_ERR_UNSUPPORTED;
        hipLaunchKernelGGL((grouped_tile_kernel<O, GATED>), dim3(static_cast<unsigned>(grid)), dim3(kPlanThreads), 0, stream, a);
        return launch_status();
    }
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
