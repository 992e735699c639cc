// The router's balance loss, per-expert counts and the gradient of the logits. The routing's weights ([Scratch] §3) train
// the experts a token chose; what keeps the router from choosing the same few is a term of its own. With p[t,:] the softmax
// of token t's logits over all E experts, n the tokens that count and f_e = counts[e] / (n K) the share of the slots:
//   loss = coef E sum_e f_e (1/n) sum_t p[t,e]
//   d_logits[t,e] = d_loss coef (E/n) p[t,e] (f_e - sum_j f_j p[t,j])      (f is piecewise constant: no gradient)
#include <algorithm>

#include "moe_common.h"

namespace moe {
namespace {

constexpr int kStatThreads = 512;
constexpr int kJoinThreads = 256, kJoinCols = 16, kMaxJoinBlocks = MOE_MAX_EXPERTS / kJoinCols;
constexpr int kBackThreads = 256;
constexpr int kMaxStatBlocks = 256;  // one a CU
constexpr int kFlush = 8;            // tokens of a lane summed in float32 before they join its double sums

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

// The sum over lanes l, l ^ 16, l ^ 32 and l ^ 48: an exchange of two registers' rows gives
// both operands.
__device__ __forceinline__ double row_sum(double v)
{
    const uint64_t w = __double_as_longlong(v);
    const uint32_t lo = static_cast<uint32_t>(w), hi = static_cast<uint32_t>(w >> 32);
    const auto a = __builtin_amdgcn_permlane16_swap(lo, lo, false, false), b = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    const double s = __longlong_as_double(static_cast<uint64_t>(b[0]) << 32 | a[0]) +
                     __longlong_as_double(static_cast<uint64_t>(b[1]) << 32 | a[1]);
    const uint64_t x = __double_as_longlong(s);
    const uint32_t xl = static_cast<uint32_t>(x), xh = static_cast<uint32_t>(x >> 32);
    const auto c = __builtin_amdgcn_permlane32_swap(xl, xl, false, false), d = __builtin_amdgcn_permlane32_swap(xh, xh, false, false);
    return __longlong_as_double(static_cast<uint64_t>(d[0]) << 32 | c[0]) +
           __longlong_as_double(static_cast<uint64_t>(d[1]) << 32 | c[1]);
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

// Column of a lane's element i of chunk q: four consecutive ones where rows are read in vectors of four.
template <int L, bool V4>
__device__ __forceinline__ int column(int sub, int q, int i)
{
    return V4 ? 4 * (sub + L * q) + i : sub + L * (4 * q + i);
}

// A token's row, 4 Q elements a lane (-inf past E).
template <int L, bool V4, int Q>
__device__ __forceinline__ void load_row(const float *__restrict__ row, int E, int sub, float (&v)[4 * Q])
{
    const float none = -__builtin_inff();
    if constexpr (V4) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = column<L, V4>(sub, q, 0);
            const u32x4 w = ld16(row + (c < E ? c : 0));
            v[4 * q] = c < E ? __uint_as_float(w.x) : none;
            v[4 * q + 1] = c < E ? __uint_as_float(w.y) : none;
            v[4 * q + 2] = c < E ? __uint_as_float(w.z) : none;
            v[4 * q + 3] = c < E ? __uint_as_float(w.w) : none;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4 * Q; ++j) {
            const int c = sub + L * j;
            const float w = row[c < E ? c : E - 1];
            v[j] = c < E ? w : none;
        }
    }
}

// The row's softmax in its place. A row whose logits are all -inf has p = 0. 2^x and 1/x by their instructions, right to an ulp:
// the exponent's roundings, of the difference, of log2 e (0.23 u) and of the product, 2.23 u (top - x) in all, are what counts. (The
// sum adds their mean over p, and as sum_j p_j (top - x_j) <= ln E that is 15.5 u at most.)
template <int L, int N>
__device__ __forceinline__ void softmax(float (&p)[N])
{
    constexpr float kLog2e = 1.44269504088896340736f;
    const float none = -__builtin_inff();
    float top = p[0];
#pragma unroll
    for (int j = 1; j < N; ++j)
        top = fmaxf(top, p[j]);
    top = token_max<L>(top);
    top = top == none ? 0.0f : top;  // exp(-inf - 0) = 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        p[j] = __builtin_amdgcn_exp2f((p[j] - top) * kLog2e);  // NaN, and +inf - +inf, stay NaN
        sum += p[j];
    }
    sum = token_sum<L>(sum);
    const float r = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
    for (int j = 0; j < N; ++j)
        p[j] *= r;
}

// ---------------------------------------------------------------- forward

struct Share {  // of an expert in a range of tokens
    float prob;
    int32_t count;
};

struct Joined {  // behind the workgroups' shares: workgroups of the join that are done, and each one's share of the loss
    int32_t done, pad;
    double dot[kMaxJoinBlocks];
};

struct StatArgs {
    const float *logits;
    const int32_t *topk_idx;
    const uint8_t *mask;
    int64_t T, tokens_per_block;
    int32_t E, K;
    float coef;
    Joined *joined;
    Share *shares;  // [blocks][E + 1]: a workgroup's, and its tokens that count
    float *loss, *prob_sum;
    int32_t *counts, *tokens;
};

// Sum over the workgroup, in every thread; the same order for the same sizes.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double *sh)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) == 0)
        sh[threadIdx.x / kWave] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w)
        s += sh[w];
    return s;
}

__device__ __forceinline__ void write_loss(const StatArgs &a, double dot, int32_t n)
{
    a.tokens[0] = n;
    const double nd = n;
    a.loss[0] = n == 0 ? 0.0f : static_cast<float>(static_cast<double>(a.coef) * a.E * dot / (nd * nd * a.K));
}

// Each workgroup takes a range of tokens, L lanes a token, two tokens at a time. A lane keeps the sums of its columns, the
// workgroup's lanes are put together in a fixed order, and the counts are integers: the results do not depend on timing.
// T16384 E256 K8 7.1 us, of which its 17 MB are 2.6: one workgroup a CU, whose wavefronts load two tokens a group of lanes, take
// their softmax and go through LDS into the workgroup's shares, one latency after the other (the slots, on their way beside the
// logits, and all columns through LDS at a time 1.9 us less). T64 E8, one launch, 3.4 us.
template <int L, bool V4, int Q>
__global__ __launch_bounds__(kStatThreads) void balance_stat_kernel(StatArgs a)
{
    constexpr int kGroups = kStatThreads / L, kWaves = kStatThreads / kWave, kCols = 4 * L, N = 4 * Q;
    __shared__ double part[kWaves][kCols * Q];
    __shared__ int32_t hist[kCols * Q];
    __shared__ int32_t ntok;
    const int sub = threadIdx.x % L, group = threadIdx.x / L, wave = threadIdx.x / kWave;
    const int64_t t0 = blockIdx.x * a.tokens_per_block, t1 = min(a.T, t0 + a.tokens_per_block);
    for (int i = threadIdx.x; i < kCols * Q; i += kStatThreads)
        hist[i] = 0;
    if (threadIdx.x == 0)
        ntok = 0;
    // a slot of this workgroup's, on its way beside the logits
    const int64_t slot = t0 * a.K + threadIdx.x, slots = t1 * a.K;
    auto counted = [&](int64_t i) { return !a.mask || a.mask[static_cast<uint32_t>(i) / static_cast<uint32_t>(a.K)]; };
    const int32_t e0 = slot < slots && counted(slot) ? a.topk_idx[slot] : -1;
    double acc[N] = {};
    int32_t mine = 0;
    if (t0 < t1) {
        float few[N] = {};
        int n = 0;
        for (int64_t t = t0 + group; t < t1; t += 2 * kGroups) {
            const int64_t u = t + kGroups;
            float p[N], q[N];
            load_row<L, V4, Q>(a.logits + t * a.E, a.E, sub, p);
            load_row<L, V4, Q>(a.logits + min(u, t1 - 1) * a.E, a.E, sub, q);
            const bool first = !a.mask || a.mask[t], second = u < t1 && (!a.mask || a.mask[min(u, t1 - 1)]);
            softmax<L>(p);
            softmax<L>(q);
#pragma unroll
            for (int j = 0; j < N; ++j)
                few[j] += (first ? p[j] : 0.0f) + (second ? q[j] : 0.0f);
            mine += first + second;
            if ((n += 2) == kFlush) {
                n = 0;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    acc[j] += static_cast<double>(few[j]);
                    few[j] = 0.0f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            acc[j] += static_cast<double>(few[j]);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const double v = L == 16 ? row_sum(acc[j]) : acc[j];
        if ((threadIdx.x & (kWave - 1)) < L)
            part[wave][column<L, V4>(sub, j / 4, j % 4)] = v;
    }
    __syncthreads();
    if (sub == 0)
        atomicAdd(&ntok, mine);
    if (e0 >= 0 && e0 < a.E)
        atomicAdd(&hist[e0], 1);
    for (int64_t i = slot + kStatThreads; i < slots; i += kStatThreads) {
        const int32_t e = a.topk_idx[i];
        if (e >= 0 && e < a.E && counted(i))
            atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    double share = 0.0;
    for (int c = threadIdx.x; c < a.E; c += kStatThreads) {
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            total += part[w][c];
        if (gridDim.x == 1) {
            a.prob_sum[c] = static_cast<float>(total);
            a.counts[c] = hist[c];
            share += hist[c] * total;
        } else {
            a.shares[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + c] = Share{static_cast<float>(total), hist[c]};
        }
    }
    if (gridDim.x == 1) {
        const double dot = block_sum<kStatThreads>(share, &part[0][0]);
        if (threadIdx.x == 0)
            write_loss(a, dot, ntok);
    } else if (threadIdx.x == 0) {
        a.shares[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + a.E] = Share{0.0f, ntok};
        if (blockIdx.x == 0)
            a.joined->done = 0;  // for the join, the next launch
    }
}

// The workgroups' sums, added in their order, kJoinCols columns a workgroup; the last one to be done has the loss. (One workgroup
// for all columns has its CU's bandwidth alone. Both launches at T16384 E256, whose shares are 0.5 MB: 13.1 us, 13.7 with 32
// columns; E1024 21.4 with 16 or 32; T4096 E128 10.0 and 9.8.) Bound by a chain of latencies.
__global__ __launch_bounds__(kJoinThreads) void balance_join_kernel(StatArgs a, int blocks)
{
    constexpr int kParts = kJoinThreads / kJoinCols, kAhead = 16;  // rows whose loads are under way together
    __shared__ double sh[kJoinThreads];
    __shared__ int32_t cnt[kJoinThreads];
    __shared__ int32_t ntok, last;
    const int col = threadIdx.x % kJoinCols, part = threadIdx.x / kJoinCols, c = blockIdx.x * kJoinCols + col;
    static_assert(kMaxStatBlocks <= kJoinThreads, "");
    const int32_t here =
        static_cast<int>(threadIdx.x) < blocks ? a.shares[static_cast<int64_t>(threadIdx.x) * (a.E + 1) + a.E].count : 0;
    if (threadIdx.x == 0)
        ntok = 0;
    double sum = 0.0;
    int32_t count = 0;
    if (c < a.E) {
        for (int b = part; b < blocks; b += kAhead * kParts) {
            Share v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                v[i] = a.shares[static_cast<int64_t>(min(b + i * kParts, blocks - 1)) * (a.E + 1) + c];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const bool there = b + i * kParts < blocks;
                sum += there ? static_cast<double>(v[i].prob) : 0.0;
                count += there ? v[i].count : 0;
            }
        }
    }
    sh[threadIdx.x] = sum;
    cnt[threadIdx.x] = count;
    __syncthreads();
    if (here)
        atomicAdd(&ntok, here);
    double share = 0.0;
    if (threadIdx.x < kJoinCols && c < a.E) {
#pragma unroll
        for (int p = 1; p < kParts; ++p) {
            sum += sh[p * kJoinCols + col];
            count += cnt[p * kJoinCols + col];
        }
        a.prob_sum[c] = static_cast<float>(sum);
        a.counts[c] = count;
        share = count * sum;
    }
    __syncthreads();
    const double dot = block_sum<kJoinThreads>(share, sh);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&a.joined->dot[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(&a.joined->done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == static_cast<int>(gridDim.x) - 1;
    }
    __syncthreads();
    if (last && threadIdx.x < kWave) {
        static_assert(kMaxJoinBlocks <= kWave, "");
        double total = 0.0;
        if (threadIdx.x < gridDim.x)
            total = __hip_atomic_load(&a.joined->dot[threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        total = wave_sum(total);
        if (threadIdx.x == 0)
            write_loss(a, total, ntok);
    }
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

// A gradient row out, with another added, which may be the row itself: each element is read before it is written, by the same lane.
template <int L, bool V4, int Q>
__device__ __forceinline__ void store_row(const float (&d)[4 * Q], const float *add, float *out, int E, int sub)
{
    if constexpr (V4) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = column<L, V4>(sub, q, 0);
            if (c >= E)
                continue;
            u32x4 b{0, 0, 0, 0};
            if (add)
                b = ld16(add + c);
            const float v[4] = {d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
            const uint32_t w[4] = {b.x, b.y, b.z, b.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = __float_as_uint(add ? v[i] + __uint_as_float(w[i]) : v[i]);
            st16(out + c, u32x4{o[0], o[1], o[2], o[3]});
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4 * Q; ++j) {
            const int c = sub + L * j;
            if (c < E)
                out[c] = add ? d[j] + add[c] : d[j];
        }
    }
}

// L lanes a token, as above; f, the same for all tokens, stays in registers. T16384 E256 with a gradient to add, 50 MB in 12-13 us;
// T2999 E61 3.7 us. With few tokens a group of lanes it is a chain of latencies: the counts one word after the other, then the
// logits, then each vector to be added.
template <int L, bool V4, int Q>
__global__ __launch_bounds__(kBackThreads) void balance_backward_kernel(BackArgs a)
{
    constexpr int kGroups = kBackThreads / L, N = 4 * Q;
    const int sub = threadIdx.x % L;
    const int32_t n = a.tokens[0];
    const float share = n > 0 ? static_cast<float>(1.0 / (static_cast<double>(n) * a.K)) : 0.0f;
    const float scale = n > 0 ? static_cast<float>(static_cast<double>(a.d_loss ? a.d_loss[0] : 1.0f) * a.coef * a.E / n) : 0.0f;
    float f[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = column<L, V4>(sub, j / 4, j % 4);
        f[j] = c < a.E ? static_cast<float>(a.counts[c]) * share : 0.0f;
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / L; t < a.T;
         t += static_cast<int64_t>(gridDim.x) * kGroups) {
        float d[N];
        load_row<L, V4, Q>(a.logits + t * a.E, a.E, sub, d);
        softmax<L>(d);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j)
            s = fmaf(f[j], d[j], s);
        s = token_sum<L>(s);
        const bool counts = n > 0 && (!a.mask || a.mask[t]);
#pragma unroll
        for (int j = 0; j < N; ++j)
            d[j] = counts ? scale * d[j] * (f[j] - s) : 0.0f;
        store_row<L, V4, Q>(d, a.add ? a.add + t * a.E : nullptr, a.out + t * a.E, a.E, sub);
    }
}

// ---------------------------------------------------------------- launches

int stat_lanes(int32_t E) { return E <= 256 ? 16 : kWave; }

// Workgroups of the forward: each has one pass over two tokens a group of lanes at least. Up to four passes one workgroup and one
// launch take less than two (T256 E64 5.9 against 7.3 us, T64 E512 6.7 against 8.1; T256 E256 10.0 against 9.2, and the host's
// launch less; T512 E64 9.0 against 7.4).
int stat_blocks(int64_t T, int32_t E)
{
    const int64_t passes = ceil_div(T, 2 * (kStatThreads / stat_lanes(E)));
    return passes <= 4 ? 1 : static_cast<int>(std::min<int64_t>(kMaxStatBlocks, passes));
}

size_t stat_bytes(int64_t T, int32_t E)
{
    const size_t blocks = static_cast<size_t>(stat_blocks(T, E));
    return blocks == 1 ? 0 : sizeof(Joined) + blocks * sizeof(Share) * (E + 1);
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
    Joined *joined = static_cast<Joined *>(workspace);
    const StatArgs a{logits, topk_idx, token_mask, T, ceil_div(T, blocks), E, K, coef, joined,
                     need > 0 ? reinterpret_cast<Share *>(joined + 1) : nullptr, loss, prob_sum, counts, tokens};
    if (E % 4 == 0 && aligned16(logits))
        MOE_BALANCE_DISPATCH(launch_stat, true, E, a, blocks, stream);
    else
        MOE_BALANCE_DISPATCH(launch_stat, false, E, a, blocks, stream);
    if (blocks > 1)
        hipLaunchKernelGGL(balance_join_kernel, dim3(static_cast<unsigned>(ceil_div(E, kJoinCols))), dim3(kJoinThreads), 0, stream, a,
                           blocks);
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
