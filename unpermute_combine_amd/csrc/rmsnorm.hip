// The residual addition with the RMS norm that stands before an MoE layer's router and dispatch, its
// output also as the FP8 rows of the FP8 dispatch, and its backward.
//
//   h[t,j] = x[t,j] + residual[t,j]          s[t] = 1 / sqrt(mean_j h[t,j]^2 + eps)
//   out[t,j] = h[t,j] * s[t] * weight[j]
// FP8, for each block of out: scale = max |out| / 448 in float32, and since s is common to the block, the codes of
//   448 h[t,j] weight[j] / max_k |h[t,k] weight[k]|
// in float64 up to one rounding to float32 and that to E4M3: neither s's rounding nor the scale's moves a code.
// Backward, g = d out, a = g * weight, m[t] = s[t]^2 * mean_j a[t,j] h[t,j]:
//   dx[t,j] = s[t] * (a[t,j] - h[t,j] * m[t]) (+ d_sum[t,j]),   dweight[j] = sum_t g[t,j] h[t,j] s[t]
//
// Otherwise everything between the loads and the one rounding of each output is float32.
#include <algorithm>
#include <cmath>

#include "moe_common.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / kWave;
constexpr float kE4M3Max = 448.0f;

__device__ __forceinline__ float load_f(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ float load_f(const float *p) { return *p; }
__device__ __forceinline__ void store_f(uint16_t *p, float v) { *p = static_cast<uint16_t>(f32_to_bf16_bits(v)); }
__device__ __forceinline__ void store_f(float *p, float v) { *p = v; }

// A row of either type behind a uniform run-time choice (weights, and the output rows).
struct Row {
    const void *p;
    bool bf16;
    __device__ __forceinline__ float operator[](int64_t i) const
    {
        return bf16 ? load_f(static_cast<const uint16_t *>(p) + i) : static_cast<const float *>(p)[i];
    }
};

struct RowOut {
    void *p;
    bool bf16;
    __device__ __forceinline__ void set(int64_t i, float v) const
    {
        if (bf16)
            store_f(static_cast<uint16_t *>(p) + i, v);
        else
            static_cast<float *>(p)[i] = v;
    }
};

// Reductions over 2 << n neighbouring lanes: within 16 lanes by DPP moves (lane xor 1, xor 2, then mirrors, which
// find the other half once its lanes agree), beyond by shuffles through LDS.
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

constexpr int kDppQuadXor1 = 0xb1, kDppQuadXor2 = 0x4e, kDppRowHalfMirror = 0x141, kDppRowMirror = 0x140;

__device__ __forceinline__ float wave_sum(float v)
{
    v += dpp<kDppQuadXor1>(v);
    v += dpp<kDppQuadXor2>(v);
    v += dpp<kDppRowHalfMirror>(v);
    v += dpp<kDppRowMirror>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

__device__ __forceinline__ float lanes_max(float v, int lanes)
{
    if (lanes > 1)
        v = fmaxf(v, dpp<kDppQuadXor1>(v));
    if (lanes > 2)
        v = fmaxf(v, dpp<kDppQuadXor2>(v));
    if (lanes > 4)
        v = fmaxf(v, dpp<kDppRowHalfMirror>(v));
    if (lanes > 8)
        v = fmaxf(v, dpp<kDppRowMirror>(v));
    if (lanes > 16)
        v = fmaxf(v, __shfl_xor(v, 16));
    if (lanes > 32)
        v = fmaxf(v, __shfl_xor(v, 32));
    return v;
}

__device__ __forceinline__ float wave_max(float v) { return lanes_max(v, kWave); }

__device__ __forceinline__ double lanes_max(double v, int lanes)
{
    for (int d = 1; d < lanes; d *= 2)
        v = fmax(v, __shfl_xor(v, d));
    return v;
}

// 1 / sqrt(v), rounded once: y, the instruction's value, one step of 2^-23 off at most, and a Newton step of it with v y in two
// floats, which leaves 2^-45 before the rounding (1 / sqrtf(v) rounds twice and is another value for every fourth v). The
// instruction does not take subnormals, so what is near them is scaled; of zero, infinity and NaN y is the value.
__device__ __forceinline__ float reciprocal_root(float v)
{
    const bool tiny = v < 0x1p-100f;
    const float u = tiny ? v * 0x1p100f : v, y = __builtin_amdgcn_rsqf(u), high = u * y, low = fmaf(u, y, -high);
    float s = fmaf(0.5f * y, fmaf(-low, y, fmaf(-high, y, 1.0f)), y);
    s = s == s ? s : y;
    return tiny ? s * 0x1p50f : s;
}

// A block's scale, and how its codes come of it.
struct BlockScale {
    float scale, to_code;
    bool ratio;  // codes by the ratio to the block's largest value; else, of zeros and near float32's subnormals, by the scale
    __device__ __forceinline__ explicit BlockScale(float amax)
        : scale(amax > 0.0f ? amax / kE4M3Max : 1.0f), to_code(__builtin_amdgcn_rcpf(scale)), ratio(amax > 0.0f && scale >= 0x1p-100f)
    {
    }
};

__device__ __forceinline__ uint2 codes8(const float (&c)[8])
{
    uint2 q;
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    q.x = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], 0, false);
    q.y = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], lo, true);
    return q;
}

// Codes of eight float32 values n = h s w, and whether all of them are sure: n and the block's largest have two roundings
// each, the scale one, its reciprocal two and the products two, 9 of 2^-24, so where 2^-20 more and less have the same code,
// that is the ratio's own. (Values that float32 rounds as subnormals have the code 0 in a block of such a scale. h s is none
// where the code is not 0 and |w| is 2^16 or less: codes begin at 2^-10 of the scale, which is 2^-100 or more, so |h s| is
// 2^-126 or more. The codes of larger weights, `large`, are not sure.)
__device__ __forceinline__ uint2 sure_codes8(const float (&n)[8], bool large, const BlockScale &b, bool &sure)
{
    const float lower = b.to_code * (1.0f - 0x1p-20f), upper = b.to_code * (1.0f + 0x1p-20f);
    float less[8], more[8];
    if (!b.ratio) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            less[j] = n[j] / b.scale;
        sure = true;
        return codes8(less);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        less[j] = n[j] * lower;
        more[j] = n[j] * upper;
    }
    const uint2 q = codes8(less), r = codes8(more);
    sure = q.x == r.x && q.y == r.y && !large;
    return q;
}

// The codes by the definition: about 1 wavefront in 100 has a value that is not sure.
__device__ __forceinline__ double max8(const float (&h)[8], const float (&w)[8])
{
    double top = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        top = fmax(top, fabs(static_cast<double>(h[j]) * static_cast<double>(w[j])));
        __builtin_amdgcn_sched_barrier(0);  // seldom run: few registers matter more than its time
    }
    return top;
}

__device__ __forceinline__ uint2 exact_codes8(const float (&h)[8], const float (&w)[8], double top)
{
    const double to_code = static_cast<double>(kE4M3Max) / top;
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        c[j] = static_cast<float>(static_cast<double>(h[j]) * static_cast<double>(w[j]) * to_code);
        __builtin_amdgcn_sched_barrier(0);
    }
    return codes8(c);
}

// Sum over the workgroup in every thread, in a fixed order.
__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float sh[kNormWaves];
    v = wave_sum(v);
    __syncthreads();  // the last call's values have been read
    if ((threadIdx.x & (kWave - 1)) == 0)
        sh[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x) / kWave; ++w)
        s += sh[w];
    return s;
}

// ---------------------------------------------------------------- forward, any length
// One workgroup per row: a pass for the sum of squares and a pass for the outputs (and with FP8
// codes one wavefront per block: its largest value, then its codes). Outputs may lie on the inputs
// element for element: each element's inputs are read by the thread that writes it, before it does.
// A thread's chain may be 2^18 elements here (like values one after the other in float32: up to 0.4% off), so it is in double.
struct NormArgs {
    const void *x, *residual;
    Row weight;
    int64_t T, H;
    float eps;
    void *sum_out;
    RowOut out;
    float *rstd;
    uint8_t *q;
    float *scales;
    int64_t block;
};

template <typename X, typename S>
__device__ __forceinline__ void norm_row(const NormArgs &a, int64_t t)
{
    const X *x = static_cast<const X *>(a.x) + t * a.H;
    const S *r = a.residual ? static_cast<const S *>(a.residual) + t * a.H : nullptr;
    S *so = a.sum_out ? static_cast<S *>(a.sum_out) + t * a.H : nullptr;
    double ss = 0.0;
    for (int64_t j = threadIdx.x; j < a.H; j += kNormThreads) {
        const double h = r ? load_f(x + j) + load_f(r + j) : load_f(x + j);
        ss = fma(h, h, ss);
    }
    const float s = reciprocal_root(block_sum(static_cast<float>(ss)) / static_cast<float>(a.H) + a.eps);
    if (a.rstd && threadIdx.x == 0)
        a.rstd[t] = s;
    if (a.q) {
        const int lane = threadIdx.x & (kWave - 1);
        const int64_t nb = a.H / a.block;
        for (int64_t b = threadIdx.x / kWave; b < nb; b += kNormWaves) {
            float amax = 0.0f;
            double top = 0.0;
            for (int64_t j = b * a.block + lane; j < (b + 1) * a.block; j += kWave) {
                const float h = r ? load_f(x + j) + load_f(r + j) : load_f(x + j), w = a.weight[j];
                amax = fmaxf(amax, fabsf(h * s * w));
                top = fmax(top, fabs(static_cast<double>(h) * static_cast<double>(w)));
            }
            const BlockScale block(wave_max(amax));
            const double to_code = static_cast<double>(kE4M3Max) / lanes_max(top, kWave);
            if (lane == 0)
                a.scales[t * nb + b] = block.scale;
            for (int64_t j = b * a.block + lane; j < (b + 1) * a.block; j += kWave) {
                const float h = r ? load_f(x + j) + load_f(r + j) : load_f(x + j), w = a.weight[j], n = h * s * w;
                const float c = block.ratio ? static_cast<float>(static_cast<double>(h) * static_cast<double>(w) * to_code)
                                            : n / block.scale;
                a.q[t * a.H + j] = static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, 0.0f, 0, false));
                if (a.out.p)
                    a.out.set(t * a.H + j, n);
                if (so)
                    store_f(so + j, h);
            }
        }
        return;
    }
    for (int64_t j = threadIdx.x; j < a.H; j += kNormThreads) {
        const float h = r ? load_f(x + j) + load_f(r + j) : load_f(x + j);
        a.out.set(t * a.H + j, h * s * a.weight[j]);
        if (so)
            store_f(so + j, h);
    }
}

template <typename X, typename S>
__global__ __launch_bounds__(kNormThreads) void add_rmsnorm_kernel(NormArgs a)
{
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
        norm_row<X, S>(a, t);
}

// ---------------------------------------------------------------- rows in registers
// 8 consecutive elements of a row of 8 or more; the address need not be aligned beyond its element (gfx950's global memory
// instructions take any), so odd lengths and offsets use the same wide accesses. Vectors past the row's end read as 0 and
// are not written.
template <typename X>
struct Raw8 {
    u32x4 v[sizeof(X) / 2];
};

// Where vector e of a row is. TAIL: the row's length is no multiple of 8; its last vector then ends with the row, and the
// elements it shares with the one before (`shared` of them) count once in sums and are stored twice, the same: one access
// in place of seven dependent ones (T16384 H7167 bf16 271 -> 208 us, backward of T8192 H7167 159 -> 115).
struct Vec {
    int at, shared;
};

template <bool TAIL>
__device__ __forceinline__ Vec vec(int e, int H)
{
    const int at = TAIL && e < H ? min(e, H - 8) : e;
    return Vec{at, e - at};
}

template <typename X>
__device__ __forceinline__ Raw8<X> load_raw(const X *row, int e, int H)
{
    Raw8<X> q{};
    if (e < H)
        __builtin_memcpy(&q, row + e, sizeof(q));
    return q;
}

__device__ __forceinline__ void widen(const Raw8<uint16_t> &q, float (&f)[8])
{
    const uint32_t u[4] = {q.v[0].x, q.v[0].y, q.v[0].z, q.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(u[i]);
        f[2 * i + 1] = bf16_hi(u[i]);
    }
}

__device__ __forceinline__ void widen(const Raw8<float> &q, float (&f)[8]) { __builtin_memcpy(f, &q, sizeof(q)); }

__device__ __forceinline__ void narrow(const float (&f)[8], Raw8<uint16_t> &q)
{
    q.v[0] = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

__device__ __forceinline__ void narrow(const float (&f)[8], Raw8<float> &q) { __builtin_memcpy(&q, f, sizeof(q)); }

template <typename X>
__device__ __forceinline__ void store8(X *row, int e, int H, const float (&f)[8])
{
    Raw8<X> q;
    narrow(f, q);
    if (e < H)
        __builtin_memcpy(row + e, &q, sizeof(q));
}

__device__ __forceinline__ void load_weight8(const Row &w, int e, int H, float (&f)[8])
{
    if (w.bf16)
        widen(load_raw(static_cast<const uint16_t *>(w.p), e, H), f);
    else
        widen(load_raw(static_cast<const float *>(w.p), e, H), f);
}

// Sum over the workgroup in every thread, in a fixed order, with one barrier: consecutive calls alternate
// between two places (`turn`), so that a wavefront still reading the last one's is not overtaken.
__device__ __forceinline__ float block_sum1(float v, int turn)
{
    __shared__ float sh[2][16];
    v = wave_sum(v);
    if ((threadIdx.x & (kWave - 1)) == 0)
        sh[turn][threadIdx.x / kWave] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < static_cast<int>(blockDim.x) / kWave; ++w)
        s += sh[turn][w];
    return s;
}

template <typename F>
__device__ __forceinline__ F block_max1(F v, int turn)
{
    __shared__ F sh[2][16];
    v = lanes_max(v, kWave);
    if ((threadIdx.x & (kWave - 1)) == 0)
        sh[turn][threadIdx.x / kWave] = v;
    __syncthreads();
    F s = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / kWave; ++w)
        s = s > sh[turn][w] ? s : sh[turn][w];
    return s;
}

// One workgroup per row, the row in registers: thread i holds the 8-element vectors i, i + blockDim, ... (NV of
// them), so that each row is read once. FP8 (kBlocks): a block of 8 << n elements lies in 1 << n neighbouring
// lanes; (kWholeRow): one scale for the row, through LDS. Memory bounds it: T16384 H7168 bf16 with a residual 163 us, 5.8
// TB/s, a large copy's rate (two passes over the row 723; workgroups that stay and have the next row's loads in flight
// 180); T1 H7168 3.0 us, a row's latency; to FP8 T8192 H7168 94 us, 4.4 TB/s, with five wavefronts a SIMD where
// the rows alone leave room for seven. Rows of more than 8192 elements are four vectors a thread, of which the compiler spills
// 19 to 34 registers to FP8 by blocks, 66 to 115 with one scale a row, up to 10 of float32 rows: T4096 H12288 bf16 78 us (5.1
// TB/s), to FP8 109 and 233, T4096 H16384 99, 125 and 266; float32 H16384 203, 254 and 368.
enum NormOut { kRows, kBlocks, kWholeRow };

template <typename X, typename S, int NV, NormOut OUT, bool TAIL>
__global__ __launch_bounds__(NV == 2 ? 512 : 1024) void add_rmsnorm_regs_kernel(NormArgs a)
{
    const int H = static_cast<int>(a.H), e0 = 8 * threadIdx.x, step = 8 * blockDim.x;
    Raw8<X> x[NV];
    Raw8<S> r[NV];
    float w[NV][8];
    const int block = static_cast<int>(a.block);
    Vec v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        v[i] = vec<TAIL>(e0 + i * step, H);
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const X *xs = static_cast<const X *>(a.x) + t * H;
        const S *rs = a.residual ? static_cast<const S *>(a.residual) + t * H : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = load_raw(xs, v[i].at, H);
            if (rs)
                r[i] = load_raw(rs, v[i].at, H);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            load_weight8(a.weight, v[i].at, H, w[i]);
        float h[NV][8];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            widen(x[i], h[i]);
            if (rs) {
                float f[8];
                widen(r[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    h[i][j] += f[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = !TAIL || j >= v[i].shared ? fmaf(h[i][j], h[i][j], ss) : ss;
        }
        bool large = false;
        if (OUT != kRows) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = fmaxf(top, fabsf(w[i][j]));
            large = top > 0x1p16f;
        }
        const float s = reciprocal_root(block_sum1(ss, turn) / static_cast<float>(H) + a.eps);
        if (a.rstd && threadIdx.x == 0)
            a.rstd[t] = s;
        if (a.sum_out) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                store8(static_cast<S *>(a.sum_out) + t * H, v[i].at, H, h[i]);
        }
        auto values = [&](int i, float (&n)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                n[j] = h[i][j] * s * w[i][j];
        };
        uint2 q[NV];
        if (OUT == kWholeRow) {
            float top = 0.0f, n[8];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                values(i, n);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = fmaxf(top, fabsf(n[j]));
            }
            const BlockScale scale(block_max1(top, turn));
            if (threadIdx.x == 0)
                a.scales[t] = scale.scale;
            bool sure = true;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                bool one;
                values(i, n);
                q[i] = sure_codes8(n, large, scale, one);
                sure = sure && one;
            }
            if (__syncthreads_or(!sure)) {
                double exact = 0.0;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    exact = fmax(exact, max8(h[i], w[i]));
                exact = block_max1(exact, turn);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    q[i] = exact_codes8(h[i], w[i], exact);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = v[i].at;
            float n[8];
            values(i, n);
            if (OUT == kBlocks) {  // H is a multiple of 8 here: no partial vectors
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    amax = fmaxf(amax, fabsf(n[j]));
                const BlockScale scale(lanes_max(amax, block / 8));
                if (e < H && e % block == 0)
                    a.scales[t * (H / block) + e / block] = scale.scale;
                bool sure;
                q[i] = sure_codes8(n, large, scale, sure);
                if (__ballot(!sure)) {
                    const uint2 exact = exact_codes8(h[i], w[i], lanes_max(max8(h[i], w[i]), block / 8));
                    q[i] = scale.ratio ? exact : q[i];
                }
            }
            if (OUT != kRows && e < H)
                __builtin_memcpy(a.q + t * H + e, &q[i], sizeof(q[i]));
            if (OUT == kRows || a.out.p) {
                if (a.out.bf16)
                    store8(static_cast<uint16_t *>(a.out.p) + t * H, e, H, n);
                else
                    store8(static_cast<float *>(a.out.p) + t * H, e, H, n);
            }
            if (OUT == kBlocks)
                __builtin_amdgcn_sched_barrier(0);  // one vector's values in registers at a time
        }
    }
}

// ---------------------------------------------------------------- backward, any length
// dx: one workgroup per row. dweight: columns by thread over ranges of rows, the ranges' sums put
// together in order by a second kernel. The threads' chains in double, as in the forward.
template <typename G, typename S, typename D>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_dx_kernel(const G *dout, const S *h, Row weight,
                                                                  const float *rstd, const D *d_sum, int64_t T, int64_t H,
                                                                  D *dx)
{
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const float s = rstd[t];
        double ah = 0.0;
        for (int64_t j = threadIdx.x; j < H; j += kNormThreads)
            ah = fma(static_cast<double>(load_f(dout + t * H + j) * weight[j]), static_cast<double>(load_f(h + t * H + j)), ah);
        const float m = s * s * (block_sum(static_cast<float>(ah)) / static_cast<float>(H));
        for (int64_t j = threadIdx.x; j < H; j += kNormThreads) {
            float v = s * fmaf(-load_f(h + t * H + j), m, load_f(dout + t * H + j) * weight[j]);
            if (d_sum)
                v += load_f(d_sum + t * H + j);
            store_f(dx + t * H + j, v);
        }
    }
}

template <typename G, typename S>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_dweight_kernel(const G *dout, const S *h, const float *rstd,
                                                                       int64_t T, int64_t H, int64_t rows, float *part)
{
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
    if (j >= H)
        return;
    const int64_t t0 = blockIdx.y * rows, t1 = min(T, t0 + rows);
    double v = 0.0;
    for (int64_t t = t0; t < t1; ++t)
        v = fma(static_cast<double>(load_f(dout + t * H + j) * rstd[t]), static_cast<double>(load_f(h + t * H + j)), v);
    part[blockIdx.y * H + j] = static_cast<float>(v);
}

// dweight = the ranges' sums put together: a workgroup takes 32 columns, its 32 rows of threads every 32nd range
// each, and the 32 partial sums meet in order. In double: there may be 2^21 ranges.
constexpr int kSumCols = 32, kSumRows = 32;

__global__ __launch_bounds__(kSumCols *kSumRows) void rmsnorm_dweight_sum_kernel(const float *part, int64_t ranges,
                                                                                  int64_t H, float *dweight)
{
    __shared__ double sh[kSumRows][kSumCols];
    const int c = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kSumCols + c;
    double v = 0.0;
    if (j < H) {
#pragma unroll 4
        for (int64_t p = g; p < ranges; p += kSumRows)
            v += part[p * H + j];
    }
    sh[g][c] = v;
    __syncthreads();
    if (g == 0 && j < H) {
        for (int k = 1; k < kSumRows; ++k)
            v += sh[k][c];
        dweight[j] = static_cast<float>(v);
    }
}

// One workgroup per row up to 2^20 of them (a grid holds fewer than 2^32 threads), then several rows each.
unsigned row_blocks(int64_t T) { return static_cast<unsigned>(T < (1 << 20) ? T : (1 << 20)); }

// Ranges of rows whose dweight sums are formed apart: 512, and more where a range would be over 1024 rows, so that no float32
// chain is longer (over 32768 rows of like values one is up to 0.05% off, over 2^22 6%).
constexpr int64_t kDwRanges = 512, kDwRows = 1024;
int64_t dw_ranges(int64_t T) { return std::min(T, std::max(kDwRanges, ceil_div(T, kDwRows))); }

// Rows in registers as in the forward: thread i keeps its columns' weights and their gradient's sums while its
// workgroup takes rows blockIdx, blockIdx + gridDim, ...; the sums of the gridDim workgroups are put together in
// order by rmsnorm_dweight_sum_kernel. Each of dout, h and d_sum is read once. T8192 H7168 bf16: 89 + 5 us, 5.3 TB/s (apart,
// with dx by rows and dweight by columns, 337); the next row's loads are in flight while a row's sum is formed. 512
// workgroups: two a CU; T16384 H4096 100 us, with 768 or 256 of them 103 and 116. Of rows of more than 8192 elements (four
// vectors a thread) two float32 operands or more spill 6 to 104 registers: T4096 H16384 bf16 114 us (4.7 TB/s), float32 255.
// Many short rows leave the chip waiting on 512 workgroups of a wavefront or two: T200000 H64 bf16 369 us, 0.28 TB/s.
template <typename G, typename S, typename D, int NV, bool TAIL>
__global__ __launch_bounds__(512) void rmsnorm_backward_regs_kernel(const G *dout, const S *h, Row weight,
                                                                     const float *rstd, const D *d_sum, int64_t T,
                                                                     int H, D *dx, float *part)
{
    const int e0 = 8 * threadIdx.x, step = 8 * blockDim.x;
    Raw8<G> gq[NV];
    Raw8<S> hq[NV];
    Raw8<D> dq[NV];
    float w[NV][8], dw[NV][8];
    int64_t t = blockIdx.x;
    Vec vs[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        vs[i] = vec<TAIL>(e0 + i * step, H);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        gq[i] = load_raw(dout + t * H, vs[i].at, H);
        hq[i] = load_raw(h + t * H, vs[i].at, H);
    }
    float s = rstd[t];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        load_weight8(weight, vs[i].at, H, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = 0.0f;
    }
    for (int turn = 0; t < T; turn ^= 1) {
        if (d_sum) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                dq[i] = load_raw(d_sum + t * H, vs[i].at, H);
        }
        float a[NV][8], x[NV][8];
        float ah = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            widen(gq[i], a[i]);
            widen(hq[i], x[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(a[i][j] * s, x[i][j], dw[i][j]);
                a[i][j] *= w[i][j];
                ah = !TAIL || j >= vs[i].shared ? fmaf(a[i][j], x[i][j], ah) : ah;
            }
        }
        const int64_t now = t;
        const float s1 = s;
        t += gridDim.x;
        if (t < T) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                gq[i] = load_raw(dout + t * H, vs[i].at, H);
                hq[i] = load_raw(h + t * H, vs[i].at, H);
            }
            s = rstd[t];
        }
        const float m = s1 * s1 * (block_sum1(ah, turn) / static_cast<float>(H));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = s1 * fmaf(-x[i][j], m, a[i][j]);
            if (d_sum) {
                float f[8];
                widen(dq[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] += f[j];
            }
            store8(dx + now * H, vs[i].at, H, v);
        }
    }
    if (part) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            store8(part + static_cast<int64_t>(blockIdx.x) * H, vs[i].at, H, dw[i]);
    }
}

// rmsnorm_dweight_sum_kernel has 32 threads a column, and a grid fewer than 2^32.
constexpr int64_t kMaxRow = 1 << 26;

// Rows of a vector or more, up to NV of them a thread, are kept in registers.
bool in_registers(int64_t H, int64_t threads, int64_t nv) { return H >= 8 && H <= 8 * nv * threads; }

bool row_type(moe_dtype d) { return d == MOE_F32 || d == MOE_BF16; }

moe_status check_norm(const void *x, moe_dtype x_dt, const void *residual, moe_dtype sum_dt, const void *weight,
                      moe_dtype weight_dt, int64_t T, int64_t H, float eps)
{
    if (x_dt == MOE_FP8_E4M3 || sum_dt == MOE_FP8_E4M3 || weight_dt == MOE_FP8_E4M3)
        return MOE_ERR_UNSUPPORTED;
    if (T < 0 || H < 1 || !(eps >= 0.0f) || std::isinf(eps) || !row_type(x_dt) || !row_type(sum_dt) ||
        !row_type(weight_dt))
        return MOE_ERR_INVALID;
    if (T > 0x7fffffff || H > kMaxRow)
        return MOE_ERR_UNSUPPORTED;
    if (T > 0 && (!x || !weight))
        return MOE_ERR_INVALID;
    return MOE_OK;
}

template <typename X, typename S, NormOut OUT, bool TAIL>
void launch_norm_regs(const NormArgs &a, hipStream_t stream)
{
    // few rows: as many threads as vectors (up to 1024), for a row's latency; many rows: two vectors a thread (T8192 H7168 to
    // FP8 with one: 127 us against 96)
    const int64_t vecs = ceil_div(a.H, 8);
    const int nv = vecs <= (a.T <= 1024 ? 1024 : 256) ? 1 : vecs <= 2 * 512 ? 2 : 4;
    const dim3 grid(row_blocks(a.T)), block(static_cast<unsigned>(ceil_div(ceil_div(vecs, nv), kWave) * kWave));
    if (nv == 1)
        hipLaunchKernelGGL((add_rmsnorm_regs_kernel<X, S, 1, OUT, TAIL>), grid, block, 0, stream, a);
    else if (nv == 2)
        hipLaunchKernelGGL((add_rmsnorm_regs_kernel<X, S, 2, OUT, TAIL>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((add_rmsnorm_regs_kernel<X, S, 4, OUT, TAIL>), grid, block, 0, stream, a);
}

bool pow2(int64_t n) { return (n & (n - 1)) == 0; }

template <typename X, typename S>
moe_status launch_norm_xs(const NormArgs &a, hipStream_t stream)
{
    const bool blocks = a.q && pow2(a.block) && a.block >= 8 && a.block <= 8 * kWave;
    if (!in_registers(a.H, 1024, 4) || (a.q && !blocks && a.block != a.H))
        hipLaunchKernelGGL((add_rmsnorm_kernel<X, S>), dim3(row_blocks(a.T)), dim3(kNormThreads), 0, stream, a);
    else if (blocks)
        launch_norm_regs<X, S, kBlocks, false>(a, stream);
    else if (a.q)
        launch_norm_regs<X, S, kWholeRow, true>(a, stream);
    else if (a.H % 8 == 0)
        launch_norm_regs<X, S, kRows, false>(a, stream);
    else
        launch_norm_regs<X, S, kRows, true>(a, stream);
    return launch_status();
}

moe_status launch_norm(const NormArgs &a, moe_dtype x_dt, moe_dtype sum_dt, hipStream_t stream)
{
    if (x_dt == MOE_BF16)
        return sum_dt == MOE_BF16 ? launch_norm_xs<uint16_t, uint16_t>(a, stream)
                                  : launch_norm_xs<uint16_t, float>(a, stream);
    return sum_dt == MOE_BF16 ? launch_norm_xs<float, uint16_t>(a, stream) : launch_norm_xs<float, float>(a, stream);
}

void launch_dweight_sum(const float *part, int64_t ranges, int64_t H, float *dweight, hipStream_t stream)
{
    hipLaunchKernelGGL(rmsnorm_dweight_sum_kernel, dim3(static_cast<unsigned>(ceil_div(H, kSumCols))),
                       dim3(kSumCols * kSumRows), 0, stream, part, ranges, H, dweight);
}

template <typename G, typename S, typename D>
moe_status launch_backward(const void *dout, const void *h, Row weight, const float *rstd, const void *d_sum,
                           int64_t T, int64_t H, void *dx, float *dweight, float *part, hipStream_t stream)
{
    const G *g = static_cast<const G *>(dout);
    const S *hs = static_cast<const S *>(h);
    const D *ds = static_cast<const D *>(d_sum);
    const int64_t vecs = ceil_div(H, 8);
    int64_t ranges = dw_ranges(T);
    if (in_registers(H, 512, 4)) {
        const int nv = vecs <= 256 ? 1 : vecs <= 2 * 512 ? 2 : 4;
        const dim3 grid(static_cast<unsigned>(ranges)), block(static_cast<unsigned>(ceil_div(ceil_div(vecs, nv), kWave) * kWave));
#define MOE_BACKWARD_LAUNCH(NV, TAIL)                                                                                  \
    hipLaunchKernelGGL((rmsnorm_backward_regs_kernel<G, S, D, NV, TAIL>), grid, block, 0, stream, g, hs, weight, rstd, \
                       ds, T, static_cast<int>(H), static_cast<D *>(dx), dweight ? part : nullptr)
        if (H % 8 == 0) {
            if (nv == 1)
                MOE_BACKWARD_LAUNCH(1, false);
            else if (nv == 2)
                MOE_BACKWARD_LAUNCH(2, false);
            else
                MOE_BACKWARD_LAUNCH(4, false);
        } else {
            if (nv == 1)
                MOE_BACKWARD_LAUNCH(1, true);
            else if (nv == 2)
                MOE_BACKWARD_LAUNCH(2, true);
            else
                MOE_BACKWARD_LAUNCH(4, true);
        }
#undef MOE_BACKWARD_LAUNCH
    } else {
        hipLaunchKernelGGL((rmsnorm_dx_kernel<G, S, D>), dim3(row_blocks(T)), dim3(kNormThreads), 0, stream, g, hs, weight,
                           rstd, ds, T, H, static_cast<D *>(dx));
        ranges = std::min(T, kDwRanges);  // of any length: their chains are in double
        if (dweight)
            hipLaunchKernelGGL((rmsnorm_dweight_kernel<G, S>),
                               dim3(static_cast<unsigned>(ceil_div(H, kNormThreads)), static_cast<unsigned>(ranges)),
                               dim3(kNormThreads), 0, stream, g, hs, rstd, T, H, ceil_div(T, ranges), part);
    }
    if (dweight)
        launch_dweight_sum(part, ranges, H, dweight, stream);
    return launch_status();
}

template <typename G, typename S>
moe_status launch_backward_d(moe_dtype dx_dt, const void *dout, const void *h, Row weight, const float *rstd,
                             const void *d_sum, int64_t T, int64_t H, void *dx, float *dweight, float *part,
                             hipStream_t stream)
{
    return dx_dt == MOE_BF16
               ? launch_backward<G, S, uint16_t>(dout, h, weight, rstd, d_sum, T, H, dx, dweight, part, stream)
               : launch_backward<G, S, float>(dout, h, weight, rstd, d_sum, T, H, dx, dweight, part, stream);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_add_rmsnorm(const void *x, moe_dtype x_dt, const void *residual, moe_dtype sum_dt,
                                      const void *weight, moe_dtype weight_dt, int64_t T, int64_t H, float eps,
                                      void *sum_out, void *out, moe_dtype out_dt, float *rstd, hipStream_t stream)
{
    using namespace moe;
    if (out_dt == MOE_FP8_E4M3)
        return MOE_ERR_UNSUPPORTED;
    const moe_status st = check_norm(x, x_dt, residual, sum_dt, weight, weight_dt, T, H, eps);
    if (st != MOE_OK)
        return st;
    if (!row_type(out_dt))
        return MOE_ERR_INVALID;
    if (T == 0)
        return MOE_OK;
    if (!out)
        return MOE_ERR_INVALID;
    return launch_norm(NormArgs{x, residual, Row{weight, weight_dt == MOE_BF16}, T, H, eps, sum_out,
                                RowOut{out, out_dt == MOE_BF16}, rstd, nullptr, nullptr, 0},
                       x_dt, sum_dt, stream);
}

extern "C" moe_status moe_add_rmsnorm_fp8(const void *x, moe_dtype x_dt, const void *residual, moe_dtype sum_dt,
                                          const void *weight, moe_dtype weight_dt, int64_t T, int64_t H, float eps,
                                          int32_t block, void *sum_out, void *out, moe_dtype out_dt, uint8_t *q,
                                          float *scales, float *rstd, hipStream_t stream)
{
    using namespace moe;
    if (out_dt == MOE_FP8_E4M3)
        return MOE_ERR_UNSUPPORTED;
    const moe_status st = check_norm(x, x_dt, residual, sum_dt, weight, weight_dt, T, H, eps);
    if (st != MOE_OK)
        return st;
    if (!row_type(out_dt) || block < 1 || H % block != 0)
        return MOE_ERR_INVALID;
    if (T == 0)
        return MOE_OK;
    if (!q || !scales)
        return MOE_ERR_INVALID;
    return launch_norm(NormArgs{x, residual, Row{weight, weight_dt == MOE_BF16}, T, H, eps, sum_out,
                                RowOut{out, out_dt == MOE_BF16}, rstd, q, scales, block},
                       x_dt, sum_dt, stream);
}

extern "C" moe_status moe_add_rmsnorm_backward_workspace_size(int64_t T, int64_t H, size_t *bytes)
{
    using namespace moe;
    if (!bytes || T < 0 || H < 1)
        return MOE_ERR_INVALID;
    if (T > 0x7fffffff || H > kMaxRow)
        return MOE_ERR_UNSUPPORTED;
    *bytes = sizeof(float) * static_cast<size_t>(dw_ranges(T) * H);
    return MOE_OK;
}

extern "C" moe_status moe_add_rmsnorm_backward(const void *dout, moe_dtype dout_dt, const void *h, moe_dtype h_dt,
                                               const void *weight, moe_dtype weight_dt, const float *rstd,
                                               const void *d_sum, int64_t T, int64_t H, void *dx, moe_dtype dx_dt,
                                               float *dweight, void *workspace, size_t workspace_bytes,
                                               hipStream_t stream)
{
    using namespace moe;
    if (dx_dt == MOE_FP8_E4M3)
        return MOE_ERR_UNSUPPORTED;
    moe_status st = check_norm(dout, dout_dt, nullptr, h_dt, weight, weight_dt, T, H, 0.0f);
    if (st != MOE_OK)
        return st;
    if (!row_type(dx_dt) || (T > 0 && (!h || !rstd || !dx)))
        return MOE_ERR_INVALID;
    if (T == 0) {  // no rows: the weight's gradient is an empty sum
        if (!dweight)
            return MOE_OK;
        launch_dweight_sum(nullptr, 0, H, dweight, stream);
        return launch_status();
    }
    size_t need = 0;
    if (dweight && (st = moe_add_rmsnorm_backward_workspace_size(T, H, &need)) != MOE_OK)
        return st;
    if (workspace_bytes < need || (need > 0 && (!workspace || !aligned16(workspace))))
        return MOE_ERR_INVALID;
    const Row w{weight, weight_dt == MOE_BF16};
    float *part = static_cast<float *>(workspace);
    if (dout_dt == MOE_BF16)
        return h_dt == MOE_BF16 ? launch_backward_d<uint16_t, uint16_t>(dx_dt, dout, h, w, rstd, d_sum, T, H, dx,
                                                                         dweight, part, stream)
                                : launch_backward_d<uint16_t, float>(dx_dt, dout, h, w, rstd, d_sum, T, H, dx, dweight,
                                                                     part, stream);
    return h_dt == MOE_BF16
               ? launch_backward_d<float, uint16_t>(dx_dt, dout, h, w, rstd, d_sum, T, H, dx, dweight, part, stream)
               : launch_backward_d<float, float>(dx_dt, dout, h, w, rstd, d_sum, T, H, dx, dweight, part, stream);
}
