// The router's balance loss, per-expert counts and the gradient of the logits. The routing's weights ([Scratch] §3) train
// the experts a token chose; what keeps the router from choosing the same few is a term of its own. With p[t,:] the softmax
// of token t's logits over all E experts, n the tokens that count and f_e = counts[e] / (n K) the share of the slots:
//   loss = coef E sum_e f_e (1/n) sum_t p[t,e]
//   d_logits[t,e] = d_loss coef (E/n) p[t,e] (f_e - sum_j f_j p[t,j])      (f is piecewise constant: no gradient)
#include <algorithm>

#include "moe_common.h"

namespace moe {
namespace {

constexpr int kStatThreads = 1024;
constexpr int kBackThreads = 256;
constexpr int kMaxStatBlocks = 128;

constexpr int kDppRowMirror = 0x140;
constexpr int kDppRowHalfMirror = 0x141;
constexpr int kDppQuadXor2 = 0x4e;
constexpr int kDppQuadXor1 = 0xb1;

template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// Over the L lanes of a token (16 or 64), in every lane of them.
template <int L>
__device__ __forceinline__ float token_max(float v)
{
    v = fmaxf(v, dpp<kDppRowMirror>(v));
    v = fmaxf(v, dpp<kDppRowHalfMirror>(v));
    v = fmaxf(v, dpp<kDppQuadXor2>(v));
    v = fmaxf(v, dpp<kDppQuadXor1>(v));
    if constexpr (L == kWave) {
        v = fmaxf(v, __shfl_xor(v, 16));
        v = fmaxf(v, __shfl_xor(v, 32));
    }
    return v;
}

template <int L>
__device__ __forceinline__ float token_sum(float v)
{
    v += dpp<kDppRowMirror>(v);
    v += dpp<kDppRowHalfMirror>(v);
    v += dpp<kDppQuadXor2>(v);
    v += dpp<kDppQuadXor1>(v);
    if constexpr (L == kWave) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}

template <int L>
__device__ __forceinline__ double token_sum(double v)
{
#pragma unroll
    for (int d = 1; d < L; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

// Column of a lane's element i of chunk q: four consecutive ones where rows are read in vectors of four.
template <int L, bool V4>
__device__ __forceinline__ int column(int sub, int q, int i)
{
    return V4 ? 4 * (sub + L * q) + i : sub + L * (4 * q + i);
}

// p of token t, 4 Q elements a lane (zeros past E). A row whose logits are all -inf has p = 0.
template <int L, bool V4, int Q>
__device__ __forceinline__ void probs(const float *__restrict__ row, int E, int sub, float (&p)[4 * Q])
{
    const float none = -__builtin_inff();
    if constexpr (V4) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = column<L, V4>(sub, q, 0);
            const u32x4 v = ld16(row + (c < E ? c : 0));
            p[4 * q] = c < E ? __uint_as_float(v.x) : none;
            p[4 * q + 1] = c < E ? __uint_as_float(v.y) : none;
            p[4 * q + 2] = c < E ? __uint_as_float(v.z) : none;
            p[4 * q + 3] = c < E ? __uint_as_float(v.w) : none;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4 * Q; ++j) {
            const int c = sub + L * j;
            const float v = row[c < E ? c : E - 1];
            p[j] = c < E ? v : none;
        }
    }
    float top = p[0];
#pragma unroll
    for (int j = 1; j < 4 * Q; ++j)
        top = fmaxf(top, p[j]);
    top = token_max<L>(top);
    top = top == none ? 0.0f : top;  // exp(-inf - 0) = 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4 * Q; ++j) {
        p[j] = expf(p[j] - top);  // NaN, and +inf - +inf, stay NaN
        sum += p[j];
    }
    sum = token_sum<L>(sum);
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < 4 * Q; ++j)
        p[j] *= r;
}

// ---------------------------------------------------------------- forward

struct StatArgs {
    const float *logits;
    const int32_t *topk_idx;
    const uint8_t *mask;
    int64_t T, tokens_per_block;
    int32_t E, K;
    float coef;
    double *psum;     // [blocks][E]: a block's sums of p
    int32_t *pcount;  // [blocks][E + 1]: its counts, and its tokens that count
    float *loss, *prob_sum;
    int32_t *counts, *tokens;
};

// Sum over the workgroup, in every thread; the same order for the same sizes.
__device__ __forceinline__ double block_sum(double v, double *sh)
{
    v = token_sum<kWave>(v);
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0)
        sh[threadIdx.x / kWave] = v;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < kStatThreads / kWave; ++w)
        s += sh[w];
    return s;
}

// The results from the sums of one column a thread (threads past E: zeros).
__device__ __forceinline__ void write_results(const StatArgs &a, int c, double sum, int32_t count, int32_t n, double *sh)
{
    if (c < a.E) {
        a.prob_sum[c] = static_cast<float>(sum);
        a.counts[c] = count;
    }
    const double dot = block_sum(c < a.E ? count * sum : 0.0, sh);
    if (threadIdx.x == 0) {
        a.tokens[0] = n;
        const double nd = n;
        a.loss[0] = n == 0 ? 0.0f : static_cast<float>(static_cast<double>(a.coef) * a.E * dot / (nd * nd * a.K));
    }
}

// Each workgroup takes a range of tokens, L lanes a token. A lane keeps the sums of its columns in double, the workgroup's
// lanes are put together in a fixed order, and the counts are integers: the results do not depend on timing.
template <int L, bool V4, int Q>
__global__ __launch_bounds__(kStatThreads) void balance_stat_kernel(StatArgs a)
{
    constexpr int kGroups = kStatThreads / L, kWaves = kStatThreads / kWave, kCols = 4 * L;
    __shared__ double part[kWaves][kCols];
    __shared__ int32_t hist[4 * L * Q];
    __shared__ int32_t ntok;
    const int sub = threadIdx.x % L, group = threadIdx.x / L, wave = threadIdx.x / kWave;
    for (int i = threadIdx.x; i < 4 * L * Q; i += kStatThreads)
        hist[i] = 0;
    if (threadIdx.x == 0)
        ntok = 0;
    __syncthreads();
    const int64_t t0 = blockIdx.x * a.tokens_per_block, t1 = min(a.T, t0 + a.tokens_per_block);
    double acc[4 * Q] = {};
    for (int64_t t = t0 + group; t < t1; t += kGroups) {
        if (a.mask && !a.mask[t])
            continue;
        float p[4 * Q];
        probs<L, V4, Q>(a.logits + t * a.E, a.E, sub, p);
#pragma unroll
        for (int j = 0; j < 4 * Q; ++j)
            acc[j] += static_cast<double>(p[j]);
        if (sub == 0)
            atomicAdd(&ntok, 1);
    }
    for (int64_t i = t0 * a.K + threadIdx.x; i < t1 * a.K; i += kStatThreads) {
        const int32_t e = a.topk_idx[i];
        if (e >= 0 && e < a.E && (!a.mask || a.mask[i / a.K]))
            atomicAdd(&hist[e], 1);
    }
    const int chunk_of = threadIdx.x;  // the thread that ends up with column threadIdx.x
    double total = 0.0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            double v = acc[4 * q + i];
            if constexpr (L == 16) {
                v += __shfl_xor(v, 16);
                v += __shfl_xor(v, 32);
            }
            if ((threadIdx.x & (kWave - 1)) < L)
                part[wave][column<L, V4>(sub, 0, i)] = v;
        }
        __syncthreads();
        if (chunk_of >= q * kCols && chunk_of < (q + 1) * kCols) {
            for (int w = 0; w < kWaves; ++w)
                total += part[w][chunk_of - q * kCols];
        }
    }
    const int32_t count = threadIdx.x < 4 * L * Q ? hist[threadIdx.x] : 0;
    const int c = threadIdx.x;
    if (gridDim.x == 1) {
        write_results(a, c, total, count, ntok, &part[0][0]);
        return;
    }
    if (c < a.E) {
        a.psum[static_cast<int64_t>(blockIdx.x) * a.E + c] = total;
        a.pcount[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + c] = count;
    }
    if (threadIdx.x == 0)
        a.pcount[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + a.E] = ntok;
}

// The workgroups' sums, added in their order, and the results.
__global__ __launch_bounds__(kStatThreads) void balance_join_kernel(StatArgs a, int blocks)
{
    __shared__ double sh[kStatThreads];
    __shared__ int32_t cnt[kStatThreads];
    __shared__ int32_t ntok;
    int width = kWave;  // threads a row of sums; the rows are dealt to kStatThreads / width of them
    while (width < a.E)
        width *= 2;
    const int c = threadIdx.x % width, part = threadIdx.x / width, parts = kStatThreads / width;
    if (threadIdx.x == 0)
        ntok = 0;
    double sum = 0.0;
    int32_t count = 0;
    if (c < a.E) {
#pragma unroll 8
        for (int b = part; b < blocks; b += parts) {
            sum += a.psum[static_cast<int64_t>(b) * a.E + c];
            count += a.pcount[static_cast<int64_t>(b) * (a.E + 1) + c];
        }
    }
    sh[threadIdx.x] = sum;
    cnt[threadIdx.x] = count;
    __syncthreads();
    if (threadIdx.x < blocks)
        atomicAdd(&ntok, a.pcount[static_cast<int64_t>(threadIdx.x) * (a.E + 1) + a.E]);
    sum = 0.0;
    count = 0;
    if (threadIdx.x < width)
        for (int p = 0; p < parts; ++p) {
            sum += sh[p * width + threadIdx.x];
            count += cnt[p * width + threadIdx.x];
        }
    __syncthreads();
    write_results(a, threadIdx.x, sum, count, ntok, sh);
}

// ---------------------------------------------------------------- backward

struct BackArgs {
    const float *logits;
    const uint8_t *mask;
    const int32_t *counts, *tokens;
    const float *d_loss, *add;
    float *out;
    int64_t T;
    int32_t E, K;
    float coef;
};

template <int L, bool V4, int Q>
__global__ __launch_bounds__(kBackThreads) void balance_backward_kernel(BackArgs a)
{
    constexpr int kGroups = kBackThreads / L;
    const int sub = threadIdx.x % L;
    const int32_t n = a.tokens[0];
    const double share = n > 0 ? 1.0 / (static_cast<double>(n) * a.K) : 0.0;
    const float scale = n > 0 ? static_cast<float>(static_cast<double>(a.d_loss ? a.d_loss[0] : 1.0f) * a.coef * a.E / n) : 0.0f;
    double f[4 * Q];
#pragma unroll
    for (int j = 0; j < 4 * Q; ++j) {
        const int c = column<L, V4>(sub, j / 4, j % 4);
        f[j] = c < a.E ? a.counts[c] * share : 0.0;
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / L; t < a.T;
         t += static_cast<int64_t>(gridDim.x) * kGroups) {
        float d[4 * Q] = {};
        if (n > 0 && (!a.mask || a.mask[t])) {
            probs<L, V4, Q>(a.logits + t * a.E, a.E, sub, d);
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < 4 * Q; ++j)
                s = fma(f[j], static_cast<double>(d[j]), s);
            s = token_sum<L>(s);
#pragma unroll
            for (int j = 0; j < 4 * Q; ++j)
                d[j] = scale * d[j] * static_cast<float>(f[j] - s);
        }
#pragma unroll
        for (int j = 0; j < 4 * Q; ++j) {
            const int c = column<L, V4>(sub, j / 4, j % 4);
            if (c < a.E)
                a.out[t * a.E + c] = a.add ? d[j] + a.add[t * a.E + c] : d[j];
        }
    }
}

// ---------------------------------------------------------------- launches

int stat_lanes(int32_t E) { return E <= 256 ? 16 : kWave; }

// Workgroups of the forward: each has one pass over its tokens at least.
int stat_blocks(int64_t T, int32_t E)
{
    return static_cast<int>(std::min<int64_t>(kMaxStatBlocks, std::max<int64_t>(1, ceil_div(T, kStatThreads / stat_lanes(E)))));
}

size_t stat_bytes(int64_t T, int32_t E)
{
    const size_t blocks = static_cast<size_t>(stat_blocks(T, E));
    return blocks == 1 ? 0 : blocks * (sizeof(double) * E + sizeof(int32_t) * (E + 1));
}

moe_status check_sizes(int64_t T, int32_t E, int32_t K, float coef)
{
    if (T < 0 || E < 1 || K < 1 || K > E || !(coef - coef == 0.0f))
        return MOE_ERR_INVALID;
    if (E > MOE_MAX_EXPERTS || K > MOE_MAX_TOPK || T > 0x7fffffff / K)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Calls FN<L, V4, Q> for E experts.
#define MOE_BALANCE_DISPATCH(FN, V4, E, ...)                   \
    do {                                                       \
        if ((E) <= 64)                                         \
            FN<16, V4, 1>(__VA_ARGS__);                        \
        else if ((E) <= 128)                                   \
            FN<16, V4, 2>(__VA_ARGS__);                        \
        else if ((E) <= 256)                                   \
            FN<16, V4, 4>(__VA_ARGS__);                        \
        else if ((E) <= 512)                                   \
            FN<kWave, V4, 2>(__VA_ARGS__);                     \
        else                                                   \
            FN<kWave, V4, 4>(__VA_ARGS__);                     \
    } while (0)

template <int L, bool V4, int Q>
void launch_stat(const StatArgs &a, int blocks, hipStream_t stream)
{
    hipLaunchKernelGGL((balance_stat_kernel<L, V4, Q>), dim3(blocks), dim3(kStatThreads), 0, stream, a);
}

template <int L, bool V4, int Q>
void launch_back(const BackArgs &a, hipStream_t stream)
{
    const int64_t blocks = std::min<int64_t>(4096, ceil_div(a.T, kBackThreads / L));
    hipLaunchKernelGGL((balance_backward_kernel<L, V4, Q>), dim3(static_cast<unsigned>(blocks)), dim3(kBackThreads), 0, stream, a);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_balance_loss_workspace_size(int64_t T, int32_t E, size_t *bytes)
{
    using namespace moe;
    if (!bytes)
        return MOE_ERR_INVALID;
    const moe_status st = check_sizes(T, E, 1, 0.0f);
    if (st != MOE_OK)
        return st;
    *bytes = stat_bytes(T, E);
    return MOE_OK;
}

extern "C" moe_status moe_balance_loss(const float *logits, const int32_t *topk_idx, const uint8_t *token_mask, int64_t T,
                                       int32_t E, int32_t K, float coef, float *loss, int32_t *counts, float *prob_sum,
                                       int32_t *tokens, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    using namespace moe;
    moe_status st = check_sizes(T, E, K, coef);
    if (st != MOE_OK)
        return st;
    if (!loss || !counts || !prob_sum || !tokens || (T > 0 && (!logits || !topk_idx)))
        return MOE_ERR_INVALID;
    const size_t need = stat_bytes(T, E);
    if (workspace_bytes < need || (need > 0 && (!workspace || !aligned16(workspace))))
        return MOE_ERR_INVALID;
    const int blocks = stat_blocks(T, E);
    double *psum = static_cast<double *>(workspace);
    const StatArgs a{logits, topk_idx, token_mask, T, ceil_div(T, blocks), E, K, coef, psum,
                     need > 0 ? reinterpret_cast<int32_t *>(psum + static_cast<size_t>(blocks) * E) : nullptr,
                     loss, prob_sum, counts, tokens};
    if (E % 4 == 0 && aligned16(logits))
        MOE_BALANCE_DISPATCH(launch_stat, true, E, a, blocks, stream);
    else
        MOE_BALANCE_DISPATCH(launch_stat, false, E, a, blocks, stream);
    if (blocks > 1)
        hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(kStatThreads), 0, stream, a, blocks);
    return launch_status();
}

extern "C" moe_status moe_balance_loss_backward(const float *logits, const uint8_t *token_mask, const int32_t *counts,
                                                const int32_t *tokens, const float *d_loss, int64_t T, int32_t E, int32_t K,
                                                float coef, const float *d_logits_in, float *d_logits, hipStream_t stream)
{
    using namespace moe;
    const moe_status st = check_sizes(T, E, K, coef);
    if (st != MOE_OK)
        return st;
    if (T == 0)
        return MOE_OK;
    if (!logits || !counts || !tokens || !d_logits)
        return MOE_ERR_INVALID;
    const BackArgs a{logits, token_mask, counts, tokens, d_loss, d_logits_in, d_logits, T, E, K, coef};
    if (E % 4 == 0 && aligned16(logits) && aligned16(d_logits) && (!d_logits_in || aligned16(d_logits_in)))
        MOE_BALANCE_DISPATCH(launch_back, true, E, a, stream);
    else
        MOE_BALANCE_DISPATCH(launch_back, false, E, a, stream);
    return launch_status();
}
