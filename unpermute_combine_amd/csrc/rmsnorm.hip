// The residual addition with the RMS norm that stands before an MoE layer's router and dispatch, its
// output also as the FP8 rows of the FP8 dispatch, and its backward.
//
//   h[t,j] = x[t,j] + residual[t,j]          s[t] = 1 / sqrt(mean_j h[t,j]^2 + eps)
//   out[t,j] = h[t,j] * s[t] * weight[j]
// FP8: the blocks of out quantized as moe_quantize_fp8 does, from the float32 values of out.
// Backward, g = d out, a = g * weight, m[t] = s[t]^2 * mean_j a[t,j] h[t,j]:
//   dx[t,j] = s[t] * (a[t,j] - h[t,j] * m[t]) (+ d_sum[t,j]),   dweight[j] = sum_t g[t,j] h[t,j] s[t]
//
// Everything between the loads and the one rounding of each output is float32.
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

__device__ __forceinline__ float wave_sum(float v)
{
    for (int off = kWave / 2; off >= 1; off >>= 1)
        v += __shfl_xor(v, off);
    return v;
}

__device__ __forceinline__ float wave_max(float v)
{
    for (int off = kWave / 2; off >= 1; off >>= 1)
        v = fmaxf(v, __shfl_xor(v, off));
    return v;
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
    float ss = 0.0f;
    for (int64_t j = threadIdx.x; j < a.H; j += kNormThreads) {
        const float h = r ? load_f(x + j) + load_f(r + j) : load_f(x + j);
        ss = fmaf(h, h, ss);
    }
    const float s = 1.0f / sqrtf(block_sum(ss) / static_cast<float>(a.H) + a.eps);
    if (a.rstd && threadIdx.x == 0)
        a.rstd[t] = s;
    if (a.q) {
        const int lane = threadIdx.x & (kWave - 1);
        const int64_t nb = a.H / a.block;
        for (int64_t b = threadIdx.x / kWave; b < nb; b += kNormWaves) {
            float amax = 0.0f;
            for (int64_t j = b * a.block + lane; j < (b + 1) * a.block; j += kWave) {
                const float h = r ? load_f(x + j) + load_f(r + j) : load_f(x + j);
                amax = fmaxf(amax, fabsf(h * s * a.weight[j]));
            }
            amax = wave_max(amax);
            const float scale = amax > 0.0f ? amax / kE4M3Max : 1.0f;
            if (lane == 0)
                a.scales[t * nb + b] = scale;
            for (int64_t j = b * a.block + lane; j < (b + 1) * a.block; j += kWave) {
                const float h = r ? load_f(x + j) + load_f(r + j) : load_f(x + j);
                const float n = h * s * a.weight[j];
                a.q[t * a.H + j] = static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(n / scale, 0.0f, 0, false));
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

// ---------------------------------------------------------------- backward, any length
// dx: one workgroup per row. dweight: columns by thread over ranges of rows, the ranges' sums put
// together in order by a second kernel.
template <typename G, typename S, typename D>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_dx_kernel(const G *dout, const S *h, Row weight,
                                                                  const float *rstd, const D *d_sum, int64_t T, int64_t H,
                                                                  D *dx)
{
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const float s = rstd[t];
        float ah = 0.0f;
        for (int64_t j = threadIdx.x; j < H; j += kNormThreads)
            ah = fmaf(load_f(dout + t * H + j) * weight[j], load_f(h + t * H + j), ah);
        const float m = s * s * (block_sum(ah) / static_cast<float>(H));
        for (int64_t j = threadIdx.x; j < H; j += kNormThreads) {
            float v = s * fmaf(-load_f(h + t * H + j), m, load_f(dout + t * H + j) * weight[j]);
            if (d_sum)
                v += load_f(d_sum + t * H + j);
            store_f(dx + t * H + j, v);
        }
    }
}

constexpr int kDwMaxRanges = 256;

template <typename G, typename S>
__global__ __launch_bounds__(kNormThreads) void rmsnorm_dweight_kernel(const G *dout, const S *h, const float *rstd,
                                                                       int64_t T, int64_t H, int64_t rows, float *part)
{
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
    if (j >= H)
        return;
    const int64_t t0 = blockIdx.y * rows, t1 = min(T, t0 + rows);
    float v = 0.0f;
    for (int64_t t = t0; t < t1; ++t)
        v = fmaf(load_f(dout + t * H + j) * rstd[t], load_f(h + t * H + j), v);
    part[blockIdx.y * H + j] = v;
}

__global__ __launch_bounds__(kNormThreads) void rmsnorm_dweight_sum_kernel(const float *part, int64_t ranges, int64_t H,
                                                                           float *dweight)
{
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
    if (j >= H)
        return;
    float v = 0.0f;
    for (int64_t p = 0; p < ranges; ++p)
        v += part[p * H + j];
    dweight[j] = v;
}

// One workgroup per row up to 2^20 of them (a grid holds fewer than 2^32 threads), then several rows each.
unsigned row_blocks(int64_t T) { return static_cast<unsigned>(T < (1 << 20) ? T : (1 << 20)); }

int64_t dw_ranges(int64_t T) { return T < kDwMaxRanges ? T : kDwMaxRanges; }

bool row_type(moe_dtype d) { return d == MOE_F32 || d == MOE_BF16; }

moe_status check_norm(const void *x, moe_dtype x_dt, const void *residual, moe_dtype sum_dt, const void *weight,
                      moe_dtype weight_dt, int64_t T, int64_t H, float eps)
{
    if (x_dt == MOE_FP8_E4M3 || sum_dt == MOE_FP8_E4M3 || weight_dt == MOE_FP8_E4M3)
        return MOE_ERR_UNSUPPORTED;
    if (T < 0 || H < 1 || !(eps >= 0.0f) || std::isinf(eps) || !row_type(x_dt) || !row_type(sum_dt) ||
        !row_type(weight_dt))
        return MOE_ERR_INVALID;
    if (T > 0x7fffffff || H > 0x7fffffffLL / 4)
        return MOE_ERR_UNSUPPORTED;
    if (T > 0 && (!x || !weight))
        return MOE_ERR_INVALID;
    return MOE_OK;
}

moe_status launch_norm(const NormArgs &a, moe_dtype x_dt, moe_dtype sum_dt, hipStream_t stream)
{
    const dim3 grid(row_blocks(a.T)), block(kNormThreads);
    if (x_dt == MOE_BF16 && sum_dt == MOE_BF16)
        hipLaunchKernelGGL((add_rmsnorm_kernel<uint16_t, uint16_t>), grid, block, 0, stream, a);
    else if (x_dt == MOE_BF16)
        hipLaunchKernelGGL((add_rmsnorm_kernel<uint16_t, float>), grid, block, 0, stream, a);
    else if (sum_dt == MOE_BF16)
        hipLaunchKernelGGL((add_rmsnorm_kernel<float, uint16_t>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((add_rmsnorm_kernel<float, float>), grid, block, 0, stream, a);
    return launch_status();
}

template <typename G, typename S, typename D>
moe_status launch_backward(const void *dout, const void *h, Row weight, const float *rstd, const void *d_sum,
                           int64_t T, int64_t H, void *dx, float *dweight, float *part, hipStream_t stream)
{
    hipLaunchKernelGGL((rmsnorm_dx_kernel<G, S, D>), dim3(row_blocks(T)), dim3(kNormThreads), 0, stream,
                       static_cast<const G *>(dout), static_cast<const S *>(h), weight, rstd,
                       static_cast<const D *>(d_sum), T, H, static_cast<D *>(dx));
    if (!dweight)
        return launch_status();
    const int64_t ranges = dw_ranges(T), rows = ceil_div(T, ranges);
    const unsigned cols = static_cast<unsigned>(ceil_div(H, kNormThreads));
    hipLaunchKernelGGL((rmsnorm_dweight_kernel<G, S>), dim3(cols, static_cast<unsigned>(ranges)), dim3(kNormThreads), 0,
                       stream, static_cast<const G *>(dout), static_cast<const S *>(h), rstd, T, H, rows, part);
    hipLaunchKernelGGL(rmsnorm_dweight_sum_kernel, dim3(cols), dim3(kNormThreads), 0, stream, part, ranges, H, dweight);
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
    if (T > 0x7fffffff || H > 0x7fffffffLL / 4)
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
        const unsigned cols = static_cast<unsigned>(ceil_div(H, kNormThreads));
        hipLaunchKernelGGL(rmsnorm_dweight_sum_kernel, dim3(cols), dim3(kNormThreads), 0, stream,
                           static_cast<const float *>(nullptr), int64_t{0}, H, dweight);
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
