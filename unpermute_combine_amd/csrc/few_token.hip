// The whole MoE layer for a few tokens, where dispatch, grouped products and combine would each be latency:
//
//   logits[t,e] = sum_j x[t,j] router[e,j]      (summed in double, rounded once to float32)
//   topk_idx, topk_w = moe_route_topk(logits)
//   h[t,k,:] = topk_w[t,k] * silu(G_e x[t]) * (U_e x[t]),  e = topk_idx[t,k],  silu(g) = g / (1 + exp(-g))
//   out[t,:] = sum_k D_e h[t,k,:] (+ bias[t,:])
//
// with expert e's gate rows G_e = w_gate_up[e][0..I), up rows U_e = w_gate_up[e][I..2I) and D_e = w_down[e].
//
// The time is that of reading the weights of the experts in use, once each (again for each further 64 tokens of an expert, or 32
// where the products do not go through LDS), and for the smallest calls that of the launches. A wavefront multiplies 32 rows of
// a weight matrix (16 of the gate's and the 16 of the up's, or 32 of the down's) by 16 or 32 tokens with MFMA 16x16 tiles: few
// tokens leave most of a tile empty, which costs nothing while the weights' stream sets the pace. The weights go from memory
// straight into the matrix instructions' operand registers, whole cache lines at a time, several loads ahead in a ring of
// registers. Measured with cold caches, of the bytes of the weights in use: T64 H7168 I1024 E256 K8 bf16 with 96 experts in use
// and up to 37 tokens on one gate and up 5.7-6.0 TB/s, down 5.0-5.4, with 221 and up to 7 on one 6.8 and 6.1; T1 of it 6.2 and
// 5.1 (plain reads of so many bytes the same way reach 6.7) in 74 us, of which 16 are router, routing, merge and launches.
#include <algorithm>

#include "moe_common.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t vec4 __attribute__((ext_vector_type(4)));

constexpr int kMaxFewTokens = MOE_MAX_FEW_TOKENS;
constexpr int kTile = 16;  // tokens and weight rows of one matrix tile

// Weight element types. A "half" is 64 bytes of each of 16 rows, 16 in each lane: the operand of the matrix instructions,
// where lane l holds row l % 16 and the (l / 16)-th quarter. A "load" is two halves, 128 bytes of each row.
enum Weights { kWF32, kWBf16, kWFp8 };
template <Weights W> constexpr int kLaneElems = W == kWF32 ? 4 : W == kWBf16 ? 8 : 16;
template <Weights W> constexpr int kHalfElems = 4 * kLaneElems<W>;
template <Weights W> constexpr int kLoadElems = 2 * kHalfElems<W>;

// The activations that meet one half of weights: as many elements, bf16 (or float32 with float32 weights).
template <Weights W>
struct Acts {
    u32x4 v[W == kWFp8 ? 2 : 1];
};

// Weights come in whole cache lines: an instruction reads 128 bytes of 8 rows, the first of two rows 0..7 and the second
// rows 8..15, and lanes 8..15 of each 16 take the second 64 bytes. This swaps lanes 8..15 of the first with lanes 0..7
// of the second (DPP moves), which leaves the two halves of all 16 rows. (Reading 64 bytes of 16 rows at once, a line is
// asked for twice: it has to stay in the 32 KB L1 meanwhile, which few enough lines in flight do.)
constexpr int kDppRowRor8 = 0x128;

__device__ __forceinline__ void swap_eights(uint32_t &a, uint32_t &b)
{
    const int x = static_cast<int>(a), y = static_cast<int>(b);
    a = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(x, y, kDppRowRor8, 0xf, 0xc, false));
    b = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(y, x, kDppRowRor8, 0xf, 0x3, false));
}

__device__ __forceinline__ void to_halves(u32x4 &a, u32x4 &b)
{
    swap_eights(a.x, b.x);
    swap_eights(a.y, b.y);
    swap_eights(a.z, b.z);
    swap_eights(a.w, b.w);
}

// 16 bytes at an even address: the aligned words that hold them (the fifth, where the address is aligned, again the
// fourth: no word is read that holds none of them), for shift_odd to put together when they have come.
__device__ __forceinline__ void load_odd(const char *p, u32x4 &v, uint32_t &over)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~uintptr_t{3};
    __builtin_memcpy(&v, reinterpret_cast<const char *>(at), sizeof(v));
    over = *reinterpret_cast<const uint32_t *>(at + 12 + 2 * (reinterpret_cast<uintptr_t>(p) & 2));
}

__device__ __forceinline__ uint32_t odd_bits(const char *p)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 2) * 8;
}

__device__ __forceinline__ void shift_odd(u32x4 &v, uint32_t over, uint32_t bits)
{
    v.x = __builtin_amdgcn_alignbit(v.y, v.x, bits);
    v.y = __builtin_amdgcn_alignbit(v.z, v.y, bits);
    v.z = __builtin_amdgcn_alignbit(v.w, v.z, bits);
    v.w = __builtin_amdgcn_alignbit(over, v.w, bits);
}

// A lane's share of a row's partial load, elements e, e + 1, ... up to len: the vector that ends with the row, zeros in
// place of the elements before e (which other lanes have). Both operands of a product are loaded so, and what counts is
// that they agree.
template <typename X, typename R>
__device__ __forceinline__ void load_tail(const X *row, int e, int len, R &r)
{
    constexpr int n = sizeof(R) / sizeof(X), words = sizeof(R) / 4, per_word = 4 / sizeof(X);
    uint32_t t[words] = {};
    if (len >= n) {
        const int at = min(e, len - n), skip = e - at;
        __builtin_memcpy(t, row + at, sizeof(t));
        // elements at .. e - 1 are another lane's; word i holds elements at + i * per_word on
#pragma unroll
        for (int i = 0; i < words; ++i) {
            const int drop = skip - i * per_word;
            t[i] = drop <= 0 ? t[i] : drop < per_word ? t[i] & 0xffff0000u : 0u;
        }
    } else {
        X v[n] = {};
#pragma unroll
        for (int i = 0; i < n - 1; ++i)
            if (e + i < len)
                v[i] = row[e + i];
        __builtin_memcpy(t, v, sizeof(t));
    }
    __builtin_memcpy(&r, t, sizeof(r));
}

template <Weights W> struct WeightType { typedef uint16_t type; };
template <> struct WeightType<kWF32> { typedef float type; };
template <> struct WeightType<kWFp8> { typedef uint8_t type; };
template <Weights W> struct ActType { typedef uint16_t type; };
template <> struct ActType<kWF32> { typedef float type; };

// Eight E4M3 codes as bf16 (exact: three mantissa bits, and the exponents of E4M3 are normal in bf16).
__device__ __forceinline__ bf16x8 fp8_to_bf16(uint32_t a, uint32_t b)
{
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// acc[token, weight row] += sum over a half's elements of act * weight. The tile's rows (A operand) are tokens and
// its columns (B operand) weight rows; both operands hold, in lane l, row or column l % 16, and the same elements in
// the same lane group and register, so any order of the elements inside a half is right.
template <Weights W>
__device__ __forceinline__ f32x4 multiply(f32x4 acc, const Acts<W> &x, const u32x4 &w)
{
    if constexpr (W == kWF32) {
        const f32x4 a = __builtin_bit_cast(f32x4, x.v[0]), b = __builtin_bit_cast(f32x4, w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], acc, 0, 0, 0);
    } else if constexpr (W == kWBf16) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.v[0]), __builtin_bit_cast(bf16x8, w),
                                                      acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.v[0]), fp8_to_bf16(w.x, w.y), acc, 0,
                                                      0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.v[1]), fp8_to_bf16(w.z, w.w), acc, 0,
                                                      0, 0);
    }
    return acc;
}

// ---------------------------------------------------------------- router
// logits = x router^T in double (matrix instructions 16x16x4): which experts are picked then does not depend on the
// order of a float32 sum, and the products of float32 or bf16 values are exact. A workgroup takes 16 experts, 16 tokens
// and one of `splits` parts of the hidden dimension, its wavefronts an equal share of that each; the parts' sums are put
// together in order where the logits are used. A launch and a chain of memory latencies: T1 H7168 E256 5.7 us, T64 9.9.
constexpr int kRouterThreads = 512, kRouterWaves = kRouterThreads / kWave;
constexpr int kRouterElems = 32;  // of a row per step: 8 in each lane group

typedef double f64x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// The wavefront's number as a value known to be the same in its lanes: which loads a wavefront takes decides branches
// around matrix instructions, and these write every lane whatever the execution mask, so the branches have to be
// scalar ones.
__device__ __forceinline__ int wave_id()
{
    return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / kWave));
}

// Parts of the hidden dimension: a workgroup for each CU, at least one step a wavefront, and no more than the routing
// sums with one wait.
constexpr int kMaxSplits = 8;

int router_splits(int64_t T, int64_t E, int64_t H)
{
    const int64_t tiles = ceil_div(T, kTile) * ceil_div(E, kTile), most = ceil_div(H, kRouterElems * kRouterWaves);
    const int64_t want = ceil_div(256, tiles);
    return static_cast<int>(std::min(std::min(want, most), int64_t{kMaxSplits}));
}

// The mine-th of `parts` parts of a tile's sums: register r of lane l holds token t0 + l / 16 + 4 r and expert e0 + l % 16.
template <typename X>
__device__ __forceinline__ f64x4 router_tile(const X *x, const X *router, int T, int H, int E, int t0, int e0, int mine,
                                             int parts)
{
    struct Elems {
        X v[8];
    };
    const int lane = threadIdx.x & (kWave - 1), m = lane % kTile, g = lane / kTile;
    const X *xr = x + static_cast<int64_t>(min(t0 + m, T - 1)) * H, *rr = router + static_cast<int64_t>(min(e0 + m, E - 1)) * H;
    const int steps = (H + kRouterElems - 1) / kRouterElems;
    const int s1 = static_cast<int64_t>(steps) * (mine + 1) / parts;
    f64x4 acc{};
    for (int s = static_cast<int64_t>(steps) * mine / parts; s < s1; ++s) {
        const int j = s * kRouterElems + g * 8;
        Elems a{}, b{};
        if (j + 8 <= H) {
            __builtin_memcpy(&a, xr + j, sizeof(a));
            __builtin_memcpy(&b, rr + j, sizeof(b));
        } else {
            load_tail(xr, j, H, a);
            load_tail(rr, j, H, b);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64(to_f32(a.v[i]), to_f32(b.v[i]), acc, 0, 0, 0);
    }
    return acc;
}

template <typename X>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(const X *x, const X *router, int T, int H, int E,
                                                                double *part)
{
    __shared__ f64x4 red[kRouterWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const int e0 = blockIdx.x * kTile, t0 = blockIdx.y * kTile;
    const int parts = gridDim.z * kRouterWaves, mine = blockIdx.z * kRouterWaves + wave;
    red[wave][lane] = router_tile(x, router, T, H, E, t0, e0, mine, parts);
    __syncthreads();
    if (threadIdx.x >= kTile * kTile)
        return;
    // neighbouring threads take neighbouring experts
    const int e = threadIdx.x % kTile, t = threadIdx.x / kTile, src = t % 4 * kTile + e, r = t / 4;
    double v = 0.0;
    for (int w = 0; w < kRouterWaves; ++w)
        v += red[w][src][r];
    if (t0 + t < T && e0 + e < E)
        part[(static_cast<int64_t>(blockIdx.z) * T + t0 + t) * E + e0 + e] = v;
}

// N logits, each the sum of its parts in order; the loads of several parts are in flight together (one after the
// other they took 37 us of a call with T = 1, E = 256).
template <int N>
__device__ __forceinline__ void logits_of(const double *part, int splits, const int (&at)[N], int64_t all, float (&out)[N])
{
    constexpr int U = N > 4 ? 2 : kMaxSplits;
    double v[N] = {};
    for (int s = 0; s < splits; s += U) {
        double p[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < N; ++n)
                p[u][n] = part[min(s + u, splits - 1) * all + at[n]];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < N; ++n)
                v[n] += s + u < splits ? p[u][n] : 0.0;
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
        out[n] = static_cast<float>(v[n]);
}

// The logits themselves, for the group-limited routing.
__global__ __launch_bounds__(kRouterThreads) void router_sum_kernel(const double *part, int splits, int all, float *logits)
{
    const int i = blockIdx.x * kRouterThreads + threadIdx.x;
    if (i >= all)
        return;
    float v[1];
    logits_of<1>(part, splits, {i}, all, v);
    logits[i] = v[0];
}

// ---------------------------------------------------------------- routing
// moe_route_topk of one token by one wavefront: lane l holds experts l, l + 64, ...; each of the K rounds takes the
// largest key of the wavefront, of equal ones that of the lowest expert. The softmax as there: double, in slot order.
// With the plan in the same launch T1 E256 K8 5.7 us; T64 8.2, and 4.9 for the plan's own launch.
constexpr int kDppQuadXor1 = 0xb1, kDppQuadXor2 = 0x4e, kDppRowHalfMirror = 0x141, kDppRowMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v)
{
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false)));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max_dpp<kDppRowMirror>(max_dpp<kDppRowHalfMirror>(max_dpp<kDppQuadXor2>(max_dpp<kDppQuadXor1>(v))));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

// The token's logits in registers, logit[j] of expert lane + 64 j.
template <int J>
__device__ __forceinline__ void select_experts(const float (&logit)[J], int t, int E, int K, int32_t *topk_idx, float *topk_w)
{
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t key[J];  // 0: no expert, or taken
#pragma unroll
    for (int j = 0; j < J; ++j)
        key[j] = lane + kWave * j < E ? orderable(logit[j]) : 0u;
    uint32_t slot_key = 0, first = 0;
    int slot_id = -1;  // of slot `lane`
    for (int k = 0; k < K; ++k) {
        uint32_t best = 0;
        int of = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool more = key[j] > best;
            best = more ? key[j] : best;
            of = more ? j : of;
        }
        const uint32_t top = wave_max(best);
        if (top == 0)  // only where logits are not numbers
            break;
        const uint64_t have = __ballot(best == top);
        int id = 0;
        if ((have & (have - 1)) == 0) {
            const int l = __builtin_ctzll(have);
            id = l + kWave * __builtin_amdgcn_readlane(of, l);
        } else {  // equal logits: the lowest id, as the largest of their complements
            id = static_cast<int>(~wave_max(best == top ? ~static_cast<uint32_t>(lane + kWave * of) : 0u));
        }
        if (k == 0)
            first = top;
        if (lane == k) {
            slot_key = top;
            slot_id = id;
        }
        if (lane == id % kWave) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j == id / kWave)
                    key[j] = 0;
        }
    }
    const double ex = lane < K ? exp(static_cast<double>(from_orderable(slot_key)) - static_cast<double>(from_orderable(first))) : 0.0;
    double z = 0.0;
    for (int k = 0; k < K; ++k)
        z += __shfl(ex, k);
    if (lane < K) {
        topk_idx[static_cast<int64_t>(t) * K + lane] = slot_id;
        topk_w[static_cast<int64_t>(t) * K + lane] = static_cast<float>(ex / z);
    }
}

template <int J>
__device__ __forceinline__ void route_token(const double *part, int splits, int T, int t, int E, int K,
                                            int32_t *topk_idx, float *topk_w)
{
    int at[J];
    float logit[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
        at[j] = t * E + min(static_cast<int>(threadIdx.x % kWave) + kWave * j, E - 1);
    logits_of<J>(part, splits, at, static_cast<int64_t>(T) * E, logit);
    select_experts<J>(logit, t, E, K, topk_idx, topk_w);
}

// ---------------------------------------------------------------- plan
// The experts in use in ascending order, and the slots s = t * K + k of each in ascending order: a stable counting
// sort by one workgroup. Each wavefront ranks its own stretch of the slots 64 at a time (the lanes that hold the same
// expert found by ballots over its bits), so the positions do not depend on timing.
struct Plan {
    int32_t *head;   // [0]: experts in use (n)
    int32_t *act;    // [n] their ids
    int32_t *start;  // [n + 1] first position of each in order
    int32_t *order;  // [start[n]] slots,
    int32_t *token;  // and the token of each
    int32_t *place;  // [T * K] each slot's position in order, -1: it routes nowhere
};

constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / kWave;

// At most 64 slots: one wavefront sorts them, a slot in each lane, by the bits of their experts from the lowest (stable).
__device__ __forceinline__ void make_small_plan(const int32_t *topk_idx, int n, int E, int K, const Plan &plan)
{
    const int lane = threadIdx.x & (kWave - 1);
    int e = lane < n ? topk_idx[lane] : E, slot = lane;
    if (e < 0 || e > E)
        e = E;  // behind every expert
    const int bits = 32 - __builtin_clz(E);
    for (int b = 0; b < bits; ++b) {
        const bool one = (e >> b) & 1;
        const uint64_t ones = __ballot(one), below = lanemask_lt();
        const int to = one ? __popcll(~ones) + __popcll(ones & below) : __popcll(~ones & below);
        e = __builtin_amdgcn_ds_permute(4 * to, e);
        slot = __builtin_amdgcn_ds_permute(4 * to, slot);
    }
    const int before = __shfl_up(e, 1);
    const bool first = e < E && (lane == 0 || before != e);
    const uint64_t firsts = __ballot(first);
    const int rank = __popcll(firsts & lanemask_lt()), routed = __popcll(__ballot(e < E));
    if (slot < n)
        plan.place[slot] = e < E ? lane : -1;
    if (e < E) {
        plan.order[lane] = slot;
        plan.token[lane] = slot / K;
    }
    if (first) {
        plan.act[rank] = e;
        plan.start[rank] = lane;
    }
    if (lane == 0) {
        plan.head[0] = __popcll(firsts);
        plan.start[__popcll(firsts)] = routed;
    }
}

__device__ __forceinline__ void make_plan(const int32_t *topk_idx, int n, int E, int K, const Plan &plan)
{
    if (n <= kWave) {
        if (threadIdx.x < kWave)
            make_small_plan(topk_idx, n, E, K, plan);
        return;
    }
    extern __shared__ uint16_t cnt[];  // [kPlanWaves][E]: each wavefront's slots per expert, then its next position
    __shared__ uint32_t wave_total[kPlanWaves];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    for (int i = threadIdx.x; i < kPlanWaves * E; i += kPlanThreads)
        cnt[i] = 0;
    __syncthreads();
    const int per = (n + kPlanThreads - 1) / kPlanThreads * kWave;
    const int s0 = wave * per, s1 = min(n, s0 + per);
    const int bits = 32 - __builtin_clz(E);  // of the ids 0..E, E standing for "no expert"
    uint16_t *mine = cnt + wave * E;
    for (int pass = 0; pass < 2; ++pass) {
        for (int s = s0; s < s1; s += kWave) {
            int e = s + lane < s1 ? topk_idx[s + lane] : E;
            if (e < 0 || e > E)
                e = E;
            uint64_t peers = ~0ull;
            for (int b = 0; b < bits; ++b) {
                const uint64_t m = __ballot((e >> b) & 1);
                peers &= ((e >> b) & 1) ? m : ~m;
            }
            const int rank = __popcll(peers & lanemask_lt());
            int pos = 0;
            if (e < E)
                pos = mine[e];
            if (pass == 1 && s + lane < s1) {
                plan.place[s + lane] = e < E ? pos + rank : -1;
                if (e < E) {
                    plan.order[pos + rank] = s + lane;
                    plan.token[pos + rank] = (s + lane) / K;
                }
            }
            __builtin_amdgcn_wave_barrier();
            if (e < E && rank == 0)
                mine[e] = static_cast<uint16_t>(pos + __popcll(peers));
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();
        if (pass == 1)
            return;
        // totals per expert, and over them the positions (low half) and the ranks of those in use (high half)
        const int e = threadIdx.x;
        uint32_t total = 0;
        if (e < E)
            for (int w = 0; w < kPlanWaves; ++w)
                total += cnt[w * E + e];
        uint32_t v = total | (total ? 1u << 16 : 0u);
        const uint32_t own = v;
        for (int off = 1; off < kWave; off <<= 1) {
            const uint32_t o = __shfl_up(v, off);
            if (lane >= off)
                v += o;
        }
        if (lane == kWave - 1)
            wave_total[wave] = v;
        __syncthreads();
        uint32_t before = 0;
        for (int w = 0; w < wave; ++w)
            before += wave_total[w];
        v += before;
        uint32_t pos = (v - own) & 0xffffu;
        if (total) {
            plan.act[(v - own) >> 16] = e;
            plan.start[(v - own) >> 16] = pos;
        }
        if (threadIdx.x == kPlanThreads - 1) {
            plan.head[0] = v >> 16;
            plan.start[v >> 16] = v & 0xffffu;
        }
        if (e < E)
            for (int w = 0; w < kPlanWaves; ++w) {
                const uint16_t c = cnt[w * E + e];
                cnt[w * E + e] = static_cast<uint16_t>(pos);
                pos += c;
            }
        __syncthreads();
    }
}

__global__ __launch_bounds__(kPlanThreads) void few_token_plan_kernel(const int32_t *topk_idx, int n, int E, int K, Plan plan)
{
    make_plan(topk_idx, n, E, K, plan);
}

// The routing of up to kPlanWaves tokens (one each wavefront) and the plan of it in one launch, of more tokens the
// routing alone, kPlanWaves tokens a workgroup.
template <int J, bool PLAN>
__global__ __launch_bounds__(kPlanThreads) void few_token_route_kernel(const double *part, int splits, int T, int E, int K,
                                                                       int32_t *topk_idx, float *topk_w, Plan plan)
{
    const int t = blockIdx.x * kPlanWaves + wave_id();
    if (t < T)
        route_token<J>(part, splits, T, t, E, K, topk_idx, topk_w);
    if (PLAN) {
        __syncthreads();  // the workgroup's own stores of topk_idx have been done
        make_plan(topk_idx, T * K, E, K, plan);
    }
}

// Router, routing and plan in one launch, for up to 16 tokens and 64 experts with little to read: one workgroup, whose
// wavefronts share the tiles of 16 experts and the hidden dimension.
constexpr int kSmallExperts = 64;

template <typename X>
__global__ __launch_bounds__(kPlanThreads) void few_token_small_route_kernel(const X *x, const X *router, int T, int H, int E,
                                                                             int K, int32_t *topk_idx, float *topk_w,
                                                                             Plan plan)
{
    __shared__ f64x4 red[kPlanWaves][kWave];
    __shared__ float logits[kTile][kSmallExperts];
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id();
    const int tiles = (E + kTile - 1) / kTile, parts = kPlanWaves / tiles;
    if (wave < tiles * parts)
        red[wave][lane] = router_tile(x, router, T, H, E, 0, wave % tiles * kTile, wave / tiles, parts);
    __syncthreads();
    const int t = threadIdx.x / kSmallExperts, e = threadIdx.x % kSmallExperts;  // 16 x 64 threads
    if (t < T && e < E) {
        double v = 0.0;
        for (int p = 0; p < parts; ++p)
            v += red[p * tiles + e / kTile][t % 4 * kTile + e % kTile][t / 4];
        logits[t][e] = static_cast<float>(v);
    }
    __syncthreads();
    if (wave < T) {
        const float logit[1] = {logits[wave][min(lane, E - 1)]};
        select_experts<1>(logit, wave, E, K, topk_idx, topk_w);
    }
    __syncthreads();  // the workgroup's own stores of topk_idx have been done
    make_plan(topk_idx, T * K, E, K, plan);
}

// ---------------------------------------------------------------- gate and up products
// A unit is 16 columns of h of one expert, 16 rows of gate and 16 of up; wavefronts take a unit each, or share the hidden
// dimension's loads of one, and then their tiles meet in LDS. h goes out in the order of the plan, already multiplied by
// the slot's weight; beside bf16 or FP8 weights as two bf16 rows whose sum it is to 16 bits, so that the down product is
// one of bf16 operands without bf16's rounding of h. Memory bounds it: T64 H7168 I1024 E256 K8 bf16 479 us, 5.9 TB/s of the
// weights in use; FP8 T8 H4096 I2048 E128 K8 69 us, 5.8; rows off the lines T133 H2056 I1399 E64 K2 102 us, 4.4.

// Registers of one load in flight.
template <Weights W, int NW, int NT, bool LO>
constexpr int kSlotRegs = 8 * (NW + NT * (LO ? 2 : 1) * (W == kWFp8 ? 2 : 1));

// How rows of weights lie and are read. kLines: they begin on cache lines, a load is a line, and each line is read by one
// instruction, past the caches (a line that two instructions share is read from memory twice that way). Others are read as
// they lie, most lines by two instructions: kWords, where they begin on 4-byte words; kOdd, where bf16 rows or their
// activations' do not (16-byte reads from there run at half the rate of those from words, so whole words are read and put
// together by shifts; FP8 rows off their words are read by kWords all the same). kWindow: a load lies in two lines, other
// bytes of them in each row, and the lines, read as with kLines, go through a window of two in LDS, a row each, from which
// the load is read wherever it begins; kWindowOdd: and the activations as with kOdd.
enum Read { kLines, kWords, kOdd, kWindow, kWindowOdd };
constexpr bool windowed(Read r) { return r == kWindow || r == kWindowOdd; }
constexpr bool odd_acts(Read r) { return r == kOdd || r == kWindowOdd; }

// LDS of the window: 16 rows of two lines, whose first 16 bytes stand behind the second line too, for what begins at its end.
// In bytes; the last 8 keep rows, whose lengths are mostly multiples of 16, in different banks (T133 H2056 I1400 E64 K2
// without them 315 us, with them 290).
constexpr int kWindowRow = 2 * 128 + 16 + 8;
template <int NW>
constexpr int kWindowBytes = NW * kTile * kWindowRow;

// The shape of a kernel: 8 wavefronts of 128 registers, of which 16 share a CU with two loads or more in flight each (8 of up
// to 256 where FP8 rows go through the window: its 70 KiB of LDS with the scales' 17 leave room for one workgroup), or
// where experts may have MANY tokens (more than a tile's) 4 of 256, of which 8 do.
template <Weights W, bool MANY>
struct Shape {
    // registers for addresses, what is being multiplied, and FP8's scales
    static constexpr int kOther = W != kWFp8 ? 40 : MANY ? 64 : 52;
    static constexpr int kRegs = (MANY ? 256 : 128) - kOther, kWaves = MANY ? 4 : 8, kThreads = kWaves * kWave;
    template <Read READ>
    static constexpr int kWavesPerSimd = MANY || (W == kWFp8 && windowed(READ)) ? 2 : 4;
    // bytes of LDS of a wavefront: its window, later its tiles
    template <Read READ>
    static constexpr int kStretch = windowed(READ) ? kWindowBytes<2> : (MANY ? 2 : 1) * 2 * kWave * 16;
};

template <Weights W, bool MANY, Read READ>
constexpr int kStretches = Shape<W, MANY>::kWaves * Shape<W, MANY>::template kStretch<READ>;

struct ExpertArgs {
    const void *x;            // [T, H] activations
    const float *topk_w;      // [T, K] or NULL
    const void *w;            // gate_up or down
    const float *scales;      // FP8
    void *h;                  // [slots][I] float32, or [slots][2][I] bf16
    float *y;                 // [slots][H]: the slots' products
    const void *bias;
    void *out;
    int T, K, H, I;
    int hI;                   // I rounded up to whole lines: the rows of h
    int nb;                   // FP8: scales per row of w,
    uint32_t per_block;       // and 2^32 over the loads of one, rounded up (0: one load each)
    int parts;                // wavefronts that share a unit's loads
    bool stagger;             // units begin with different loads
    bool tiled;               // experts with many tokens take the tiled product
    bool out_bf16;
    Plan plan;
};

// FP8: the scales of NW rows of weights (one per lane column). They come for 16 loads at a time, 16 of a row side by side,
// are kept in registers until the wavefront is there, and are read from LDS load by load. (One load's at a time, each
// instruction would ask for a cache line per row: T8 H4096 I2048 E128 K8 with 51 experts in use 273 -> 221 us.)
constexpr int kScaleLoads = 16, kScaleStride = kScaleLoads + 1;  // the stride keeps rows in different banks
template <Weights W, int NW>
constexpr int kScaleFloats = W == kWFp8 ? NW * kTile * kScaleStride : 1;  // of LDS per wavefront

template <int NW>
struct Scales {
    const float *row[NW];
    int nb, last;        // scales of a row, rows there are but one
    uint32_t per_block;  // 2^32 over the loads of one scale, rounded up (0: one load each)
    float *lds;          // the wavefront's
    float next[4 * NW];
    int l0, n, left, at;  // loads l0 .. l0 + n - 1; of the 16 in LDS, not yet used; the first of those in `next`

    __device__ __forceinline__ void fetch()
    {
        const int lane = threadIdx.x & (kWave - 1), l = l0 + min(at + lane % kTile, n - 1);
        const int block = per_block ? __umulhi(l, per_block) : l;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < NW; ++i)
                next[4 * i + q] = row[i][min(4 * q + lane / kTile, last) * nb + block];
    }

    // The first load used will be l0 + first; beyond 16 loads, first is a multiple of 16.
    __device__ __forceinline__ void begin(int from, int loads, int first)
    {
        l0 = from;
        n = loads;
        left = 0;
        at = first & -kScaleLoads;
        fetch();
    }

    // Before each load, in order (beyond the last one the first follows).
    __device__ __forceinline__ void step()
    {
        if (left == 0) {
            const int lane = threadIdx.x & (kWave - 1);
            // the wavefront's own LDS operations are done in order: this only keeps the compiler from moving them
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    lds[(i * kTile + 4 * q + lane / kTile) * kScaleStride + lane % kTile] = next[4 * i + q];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            left = n <= kScaleLoads ? n : min(kScaleLoads, n - at);
            at = at + kScaleLoads < n ? at + kScaleLoads : 0;
            if (n > kScaleLoads)
                fetch();
        }
        --left;
    }

    // Of load l and weight row i.
    __device__ __forceinline__ float of(int l, int i) const
    {
        return lds[(i * kTile + static_cast<int>(threadIdx.x % kTile)) * kScaleStride + ((l - l0) & (kScaleLoads - 1))];
    }
};

// NW rows of weights (one per lane column) as they stream through a wavefront. Addresses are a uniform base, which
// moves, and a 32-bit offset in each lane, which does not.
template <Weights W, int NW, Read READ>
struct WeightRows {
    typedef typename WeightType<W>::type Wt;
    const char *w[NW];
    uint32_t w_row;
    uint32_t w_off[windowed(READ) ? NW : 1][2];
    // windowed: offsets from row 0's line; the first and last 16-byte word that holds a byte of the row
    uint32_t low[NW][2], high[NW][2];
    uint32_t at[NW];  // of the lane's share of load 0 in its row of the window
    char *window;
    Scales<NW> scales;  // FP8

    struct Load {
        u32x4 w[NW][2];
        uint32_t over[NW][2];  // kOdd
    };

    // Rows 0..15 from w[] on, of len elements each; rows past `last` are read as that one.
    __device__ __forceinline__ void rows_of(int len, int last, char *lds)
    {
        const int lane = threadIdx.x & (kWave - 1), m = lane % kTile, g = lane / kTile, chunk = m / 8 * 4 + g;
        const uint32_t bytes = static_cast<uint32_t>(len) * sizeof(Wt);
        w_row = min(m, last) * bytes;
        window = lds;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t row = min(8 * h + m % 8, last) * bytes;
            if constexpr (!windowed(READ)) {
                w_off[0][h] = row + 16 * chunk;
            } else {
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const uint32_t from = row + in_line(w[i]);
                    w_off[i][h] = (from & ~127u) + 16 * chunk;
                    low[i][h] = from & ~15u;
                    high[i][h] = (from + bytes - 1) & ~15u;
                }
            }
        }
        if constexpr (windowed(READ))
#pragma unroll
            for (int i = 0; i < NW; ++i)
                at[i] = ((in_line(w[i]) + w_row) & 127u) + 16 * g;
    }

    __device__ __forceinline__ static uint32_t in_line(const char *p) { return reinterpret_cast<uintptr_t>(p) & 127u; }

    __device__ __forceinline__ void scales_of(const ExpertArgs &a, int last, float *lds)
    {
        scales.nb = a.nb;
        scales.last = last;
        scales.per_block = a.per_block;
        scales.lds = lds + wave_id() * kScaleFloats<W, NW>;
    }

    __device__ __forceinline__ static void load_word(const char *p, u32x4 &v)
    {
        const vec4 n = __builtin_nontemporal_load(reinterpret_cast<const vec4 *>(p));
        v = u32x4{n.x, n.y, n.z, n.w};
    }

    // Windowed: line l of the rows.
    __device__ __forceinline__ void issue_line(Load &q, int l) const
    {
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t off = min(max(w_off[i][h] + 128 * l, low[i][h]), high[i][h]);
                load_word(w[i] - in_line(w[i]) + off, q.w[i][h]);
            }
    }

    __device__ __forceinline__ void issue(Load &q, int l) const
    {
        if constexpr (windowed(READ)) {
            issue_line(q, l + 1);
        } else {
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const char *p = w[i] + static_cast<int64_t>(l) * 128 + w_off[0][h];
                    if constexpr (READ == kLines)
                        load_word(p, q.w[i][h]);
                    else if constexpr (READ == kOdd)
                        load_odd(p, q.w[i][h], q.over[i][h]);
                    else
                        __builtin_memcpy(&q.w[i][h], p, sizeof(q.w[i][h]));
                }
        }
    }

    // Windowed: line l, which has come, into the window. (The wavefront's own LDS operations are done in order: the fences only
    // keep the compiler from moving them.)
    __device__ __forceinline__ void put_line(const Load &q, int l) const
    {
        const int lane = threadIdx.x & (kWave - 1), m = lane % kTile, chunk = m / 8 * 4 + lane / kTile;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                char *row = window + (i * kTile + 8 * h + m % 8) * kWindowRow;
                __builtin_memcpy(__builtin_assume_aligned(row + (l & 1) * 128 + 16 * chunk, 8), &q.w[i][h], 16);
                if ((l & 1) == 0 && chunk == 0)
                    __builtin_memcpy(__builtin_assume_aligned(row + 256, 8), &q.w[i][h], 16);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }

    // Load l, which has come, made into the matrix instructions' operands.
    __device__ __forceinline__ void arrange(Load &q, int l) const
    {
        if constexpr (windowed(READ)) {
            put_line(q, l + 1);
            const int m = threadIdx.x % kTile;
#pragma unroll
            for (int i = 0; i < NW; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t from = (at[i] + 64 * h + (l & 1) * 128) & 255u;
                    const uint32_t *p = reinterpret_cast<const uint32_t *>(window + (i * kTile + m) * kWindowRow + (from & ~3u));
                    q.w[i][h] = u32x4{p[0], p[1], p[2], p[3]};
                    if (W != kWF32)
                        shift_odd(q.w[i][h], p[4], (from & 3u) * 8);
                }
        } else {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                if constexpr (READ == kOdd) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        shift_odd(q.w[i][h], q.over[i][h], odd_bits(w[i] + w_off[0][h]));
                }
                to_halves(q.w[i][0], q.w[i][1]);
            }
        }
    }

    // The rows' partial load, from element `whole` of len on, as operands.
    __device__ __forceinline__ void tail(Load &q, int whole, int len) const
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NW; ++i)
                load_tail(reinterpret_cast<const Wt *>(w[i] + w_row),
                          whole + h * kHalfElems<W> + static_cast<int>(threadIdx.x % kWave / kTile) * kLaneElems<W>, len,
                          q.w[i][h]);
    }
};

// acc[i] += tile of activations * weight rows i, one half of a load.
template <Weights W, int NW>
__device__ __forceinline__ void multiply_rows(f32x4 (&acc)[NW], const Acts<W> &x, const u32x4 (&w)[NW][2], int h)
{
#pragma unroll
    for (int i = 0; i < NW; ++i)
        acc[i] = multiply<W>(acc[i], x, w[i][h]);
}

// The products of NW rows of weights with NT tiles of 16 tokens over a range of loads: LO adds the activations' second
// bf16 row, `lo` bytes behind the first. The loads run D ahead of the matrix instructions in a ring of registers, so
// that each wavefront keeps 2 * D * NW KiB of weights in flight all the time.
template <Weights W, int NW, int NT, bool LO, int REGS, Read READ>
struct Product {
    typedef WeightRows<W, NW, READ> Rows;
    typedef typename Rows::Wt Wt;
    typedef typename ActType<W>::type X;
    // 4, 2 or 1: most rows and parts of them are an even number of loads, and three at a time leave one over (T4 H2048
    // I1024 K4, gate and up: 36 us with three, 29 with two). Through the window two at most (T30 H2057 I1399 E64 K4 with four
    // 228 us, two 201, one 197; T64 H7170 I1026 E64 K8 with two 567, one 584)
    static constexpr int kRoom = (REGS - 4 * NW * NT) / kSlotRegs<W, NW, NT, LO>;
    static constexpr int D = kRoom >= 4 && !windowed(READ) ? 4 : kRoom >= 2 ? 2 : 1;
    static constexpr int kActBytes = kHalfElems<W> * sizeof(X);  // of a token's row per half
    Rows rows;
    const char *x;
    uint32_t x_row[NT];
    int64_t lo;
    f32x4 acc[NT][NW];

    struct Slot {
        typename Rows::Load w;
        Acts<W> x[NT][2], y[NT][2];
        uint32_t x_over[NT][2];  // odd_acts
    };

    __device__ __forceinline__ void multiply_slot(const Slot &q, const float (&scale)[NW])
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 p[NW];
#pragma unroll
            for (int i = 0; i < NW; ++i)
                p[i] = W == kWFp8 ? f32x4{} : acc[t][i];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                multiply_rows<W, NW>(p, q.x[t][h], q.w.w, h);
                if (LO)
                    multiply_rows<W, NW>(p, q.y[t][h], q.w.w, h);
            }
#pragma unroll
            for (int i = 0; i < NW; ++i)
                acc[t][i] = W == kWFp8 ? acc[t][i] + p[i] * scale[i] : p[i];  // a load lies in one block of scales
        }
    }

    __device__ __forceinline__ void add(Slot &q, int l)
    {
        float scale[NW] = {};
        if (W == kWFp8) {
            rows.scales.step();
#pragma unroll
            for (int i = 0; i < NW; ++i)
                scale[i] = rows.scales.of(l, i);
        }
        rows.arrange(q.w, l);
        if constexpr (odd_acts(READ) && !LO) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    shift_odd(q.x[t][h].v[0], q.x_over[t][h], odd_bits(x + x_row[t]));
        }
        multiply_slot(q, scale);
    }

    __device__ __forceinline__ void issue_acts(Slot &q, int l)
    {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t off = x_row[t] + kActBytes / 4 * (threadIdx.x % kWave / kTile);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char *row = x + static_cast<int64_t>(2 * l + h) * kActBytes;
                if constexpr (odd_acts(READ) && !LO) {
                    load_odd(row + off, q.x[t][h].v[0], q.x_over[t][h]);
                } else {
                    __builtin_memcpy(&q.x[t][h], row + off, sizeof(q.x[t][h]));
                    if (LO)
                        __builtin_memcpy(&q.y[t][h], row + lo + off, sizeof(q.y[t][h]));
                }
            }
        }
    }

    // Loads l0 .. l1 - 1 of rows of len elements, beginning with the turn-th of them (FP8: where they are more than 16, the
    // turn-th 16; windowed: the first).
    __device__ __forceinline__ void run(int l0, int l1, int len, int turn)
    {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < NW; ++i)
                acc[t][i] = f32x4{};
        const int whole = min(l1, len / kLoadElems<W>), n = whole - l0;
        if (n > 0) {
            Slot q[D];
            const bool sixteens = W == kWFp8 && n > kScaleLoads;
            const int skip = sixteens ? turn % ((n + kScaleLoads - 1) / kScaleLoads) * kScaleLoads : turn % n;
            int at = windowed(READ) ? l0 : l0 + skip, use = at, first[D];
            const int last = at == l0 ? whole - 1 : at - 1;
            auto next = [&] { at = at == last ? at : at == whole - 1 ? l0 : at + 1; };
            auto multiply_next = [&](Slot &s) {
                add(s, use);
                use = use == whole - 1 ? l0 : use + 1;
            };
            if (W == kWFp8)
                rows.scales.begin(l0, n, at - l0);
            typename Rows::Load line;
            if constexpr (windowed(READ))
                rows.issue_line(line, l0);
#pragma unroll
            for (int u = 0; u < D; ++u) {  // weights first: the activations' addresses are longer in coming
                first[u] = at;
                rows.issue(q[u].w, at);
                next();
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < D; ++u)
                issue_acts(q[u], first[u]);
            if constexpr (windowed(READ))
                rows.put_line(line, l0);
            int l = 0;
            for (; l + D < n; l += D) {
#pragma unroll
                for (int u = 0; u < D; ++u) {
                    multiply_next(q[u]);
                    rows.issue(q[u].w, at);
                    issue_acts(q[u], at);
                    next();
                    __builtin_amdgcn_sched_barrier(0);  // left alone, the scheduler gathers the loop's loads at its end
                }
            }
#pragma unroll
            for (int u = 0; u < D; ++u)
                if (l + u < n)
                    multiply_next(q[u]);
        }
        if (W != kWFp8 && whole < l1) {  // the row's last load, partial
            Slot z;
            rows.tail(z.w, whole * kLoadElems<W>, len);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = (2 * whole + h) * kHalfElems<W> + static_cast<int>(threadIdx.x % kWave / kTile) * kLaneElems<W>;
                    load_tail(reinterpret_cast<const X *>(x + x_row[t]), e, len, z.x[t][h]);
                    if (LO)
                        load_tail(reinterpret_cast<const X *>(x + x_row[t] + lo), e, len, z.y[t][h]);
                }
            multiply_slot(z, {});
        }
    }
};

// The products of two rows of weights a lane column with NT tiles of tokens, for a workgroup of 4 wavefronts with
// different weight rows and the same tokens: per load the tokens' activations go through LDS once for all wavefronts
// (two buffers, one barrier a load), where every wavefront alone would fetch each of them from L2 (T256 H4096 I2048 E16 K4,
// 64 tokens an expert: gate and up 290 -> 219 us, down 233 -> 148).
template <Weights W, int NT, bool LO, Read READ>
struct TiledProduct {
    typedef WeightRows<W, 2, READ> Rows;
    typedef typename ActType<W>::type X;
    static constexpr int kThreads = 4 * kWave, kRowChunks = W == kWFp8 ? 16 : 8, kPlanes = LO ? 2 : 1;
    static constexpr int kPlaneChunks = NT * kTile * kRowChunks, kChunks = kPlaneChunks * kPlanes;  // of 16 bytes
    static constexpr int Q = kChunks / kThreads;  // chunks a thread carries
    static constexpr int kBytes = 2 * kChunks * 16;
    // loads in flight: what the registers beside the accumulators hold, eight at most
    static constexpr int kRoom = (W == kWFp8 ? 110 : 160) / (16 + 4 * Q), D = kRoom > 8 ? 8 : kRoom;
    static constexpr int kPerLane = kRowChunks / 8;  // chunks of a lane's share of a half
    Rows rows;
    const char *x;
    int64_t lo;
    f32x4 acc[2][NT];

    struct Slot {
        typename Rows::Load w;
        vec4 x[Q];  // of the load after w's
    };

    // Chunk c of row r, with the rows' chunks permuted so that neighbouring rows' are in different banks.
    __device__ __forceinline__ static int place(int plane, int r, int c)
    {
        return plane * kPlaneChunks + r * kRowChunks + (c ^ (r & 7));
    }

    __device__ __forceinline__ void multiply_load(const u32x4 *buf, const typename Rows::Load &q, const float (&scale)[2])
    {
        const int lane = threadIdx.x & (kWave - 1), m = lane % kTile, g = lane / kTile;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4 p[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p[i] = W == kWFp8 ? f32x4{} : acc[i][t];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int pl = 0; pl < kPlanes; ++pl) {
                    Acts<W> a;
#pragma unroll
                    for (int i = 0; i < kPerLane; ++i)
                        a.v[i] = buf[place(pl, t * kTile + m, h * (kRowChunks / 2) + g * kPerLane + i)];
                    multiply_rows<W, 2>(p, a, q.w, h);
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                acc[i][t] = W == kWFp8 ? acc[i][t] + p[i] * scale[i] : p[i];
        }
    }

    // All loads of rows of len elements; row_of(r) is the byte offset of the r-th token's row from x.
    template <typename F>
    __device__ __forceinline__ void run(int len, u32x4 *lds, F row_of)
    {
        uint32_t from[Q];
        int to[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int j = threadIdx.x + i * kThreads, r = j / kRowChunks % (NT * kTile), c = j % kRowChunks;
            from[i] = row_of(r) + 16 * c;
            to[i] = place(j / kPlaneChunks, r, c);
        }
        auto plane_of = [&](int i) { return x + (LO && i >= Q / 2 ? lo : 0); };
        auto issue_x = [&](vec4 (&v)[Q], int l) {
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                vec4 n;
                __builtin_memcpy(&n, plane_of(i) + static_cast<int64_t>(l) * kRowChunks * 16 + from[i], 16);
                v[i] = n;
            }
        };
        auto stage = [&](const vec4 (&v)[Q], int b) {
#pragma unroll
            for (int i = 0; i < Q; ++i)
                reinterpret_cast<vec4 *>(lds)[b * kChunks + to[i]] = v[i];
        };
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                acc[i][t] = f32x4{};
        const int n = len / kLoadElems<W>;
        int b = 0;
        if (n > 0) {
            Slot q[D];
            vec4 x0[Q];
            if (W == kWFp8)
                rows.scales.begin(0, n, 0);
            issue_x(x0, 0);
#pragma unroll
            for (int u = 0; u < D; ++u) {
                rows.issue(q[u].w, min(u, n - 1));
                issue_x(q[u].x, min(u + 1, n - 1));
            }
            stage(x0, 0);
            for (int l = 0; l < n; l += D) {
#pragma unroll
                for (int u = 0; u < D; ++u) {
                    if (l + u < n) {
                        __syncthreads();
                        float scale[2] = {};
                        if (W == kWFp8) {
                            rows.scales.step();
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                scale[i] = rows.scales.of(l + u, i);
                        }
                        rows.arrange(q[u].w, l + u);
                        multiply_load(lds + b * kChunks, q[u].w, scale);
                        b ^= 1;
                        stage(q[u].x, b);
                        rows.issue(q[u].w, min(l + u + D, n - 1));
                        issue_x(q[u].x, min(l + u + D + 1, n - 1));
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
        if (W != kWFp8 && n * kLoadElems<W> < len) {  // the last load, partial
            vec4 v[Q];
            typename Rows::Load z;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int c = (threadIdx.x + i * kThreads) % kRowChunks;
                load_tail(reinterpret_cast<const X *>(plane_of(i) + from[i] - 16 * c), n * kLoadElems<W> + c * kLaneElems<W>,
                          len, v[i]);
            }
            rows.tail(z, n * kLoadElems<W>, len);
            __syncthreads();
            stage(v, b);
            __syncthreads();
            multiply_load(lds + b * kChunks, z, {});
        }
        __syncthreads();  // the buffers are free again
    }
};

// How a workgroup's wavefronts divide its work: `parts` of them (a power of two) share the loads of one unit of 16 or
// 32 weight rows, the others take other units.
struct Share {
    int unit, part;
    __device__ __forceinline__ Share(int waves, int parts)
    {
        const int wave = wave_id();
        unit = blockIdx.x * (waves / parts) + wave / parts;
        part = wave & (parts - 1);
    }
};

// The parts' tiles put together in order, f(unit, tile row, column, sums of the two weight rows). Register r of lane l
// holds the tile's row 4 (l / 16) + r and column l % 16.
template <int WAVES, int NT, int STRIDE, typename F>
__device__ __forceinline__ void join_parts(const f32x4 (&acc)[NT][2], int parts, char *lds, F f)
{
    constexpr int values = NT * kTile * kTile;
    const int lane = threadIdx.x & (kWave - 1);
    auto tile = [&](int wave, int t, int i) {  // each wavefront's own stretch of LDS holds its tiles
        return reinterpret_cast<f32x4 *>(lds + wave * STRIDE) + (t * 2 + i) * kWave;
    };
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            tile(wave_id(), t, i)[lane] = acc[t][i];
    __syncthreads();
    for (int i = threadIdx.x; i < WAVES / parts * values; i += WAVES * kWave) {
        const int first = i / values * parts, t = i % values / (kTile * kTile), v = i % (kTile * kTile);
        // neighbouring threads take neighbouring columns
        const int row = v / kTile, col = v % kTile, src = row / 4 * kTile + col, r = row % 4;
        float sum[2] = {};
        for (int w = first; w < first + parts; ++w)
#pragma unroll
            for (int n = 0; n < 2; ++n)
                sum[n] += tile(w, t, n)[src][r];
        f(first / parts, t * kTile + row, col, sum);
    }
    __syncthreads();
}

// The plan's entry of the expert that a workgroup takes; its entries are read together, before it is known whether
// there is such an expert (the arrays have them).
struct Entry {
    int64_t ex;
    int p0, n;
    __device__ __forceinline__ Entry(const Plan &plan, int i)
    {
        const int used = plan.head[0];
        ex = plan.act[i];
        p0 = plan.start[i];
        n = i < used ? plan.start[i + 1] - p0 : 0;
    }
};

// The weight rows of a gate and up unit: 16 columns of h. Columns past the last one take its place: what they give is
// not stored.
template <Weights W, Read READ>
__device__ __forceinline__ void gate_up_weights(const ExpertArgs &a, const Entry &en, int unit, char *window, float *scales,
                                                WeightRows<W, 2, READ> &rows)
{
    const int c0 = min(unit * kTile, a.I - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // the gate's rows, the up's rows
        const int64_t row = (en.ex * 2 + i) * a.I + c0;
        rows.w[i] = static_cast<const char *>(a.w) + row * a.H * sizeof(typename WeightType<W>::type);
        rows.scales.row[i] = a.scales + row * a.nb;
    }
    rows.rows_of(a.H, a.I - 1 - c0, window);
    rows.scales_of(a, a.I - 1 - c0, scales);
}

// h of the expert's token `row`, column c.
template <Weights W>
__device__ __forceinline__ void store_h(const ExpertArgs &a, const Entry &en, int row, int c, float gate, float up)
{
    if (row >= en.n || c >= a.I)
        return;
    const int pos = en.p0 + row;
    const float weight = a.topk_w ? a.topk_w[a.plan.order[pos]] : 1.0f;
    const float h = gate / (1.0f + expf(-gate)) * up * weight;
    if (W == kWF32) {
        static_cast<float *>(a.h)[static_cast<int64_t>(pos) * a.hI + c] = h;
    } else {
        uint16_t *hr = static_cast<uint16_t *>(a.h) + static_cast<int64_t>(pos) * 2 * a.hI;
        const uint32_t hi = f32_to_bf16_bits(h);
        const float rest = h - __uint_as_float(hi << 16);
        hr[c] = static_cast<uint16_t>(hi);
        // an infinite or NaN h is wholly in the first row
        hr[a.hI + c] = (hi & 0x7f80u) == 0x7f80u ? 0 : static_cast<uint16_t>(f32_to_bf16_bits(rest));
    }
}

// Up to NT tiles of an expert's tokens, from row r0 on.
template <Weights W, int NT, typename Sh, Read READ>
__device__ __forceinline__ void gate_up_stream(const ExpertArgs &a, const Entry &en, int r0, char *lds, float *scales)
{
    Product<W, 2, NT, false, Sh::kRegs, READ> p;
    const Share my(Sh::kWaves, a.parts);
    gate_up_weights<W, READ>(a, en, my.unit, lds + wave_id() * Sh::template kStretch<READ>, scales, p.rows);
    p.lo = 0;
    p.x = static_cast<const char *>(a.x);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = min(r0 + t * kTile + static_cast<int>(threadIdx.x % kTile), en.n - 1);
        p.x_row[t] = static_cast<uint32_t>(a.plan.token[en.p0 + r] * a.H) * sizeof(typename ActType<W>::type);
    }
    const int loads = (a.H + kLoadElems<W> - 1) / kLoadElems<W>;
    p.run(loads * my.part / a.parts, loads * (my.part + 1) / a.parts, a.H, a.stagger ? my.unit : 0);
    join_parts<Sh::kWaves, NT, Sh::template kStretch<READ>>(p.acc, a.parts, lds,
                                                            [&](int unit, int row, int column, const float (&v)[2]) {
        store_h<W>(a, en, r0 + row, (blockIdx.x * (Sh::kWaves / a.parts) + unit) * kTile + column, v[0], v[1]);
    });
}

// The same with the tokens' rows through LDS; the workgroup's wavefronts take a unit each.
template <Weights W, int NT, Read READ>
__device__ __forceinline__ void gate_up_tiles(const ExpertArgs &a, const Entry &en, int r0, char *lds, float *scales)
{
    TiledProduct<W, NT, false, READ> p;
    const int unit = blockIdx.x * 4 + wave_id(), lane = threadIdx.x & (kWave - 1);
    gate_up_weights<W, READ>(a, en, unit, nullptr, scales, p.rows);
    p.lo = 0;
    p.x = static_cast<const char *>(a.x);
    p.run(a.H, reinterpret_cast<u32x4 *>(lds), [&](int r) {
        return static_cast<uint32_t>(a.plan.token[en.p0 + min(r0 + r, en.n - 1)] * a.H) *
               static_cast<uint32_t>(sizeof(typename ActType<W>::type));
    });
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            store_h<W>(a, en, r0 + t * kTile + lane / kTile * 4 + r, unit * kTile + lane % kTile, p.acc[0][t][r], p.acc[1][t][r]);
}

// LDS of a kernel: the wavefronts' stretches, or the activations of the largest tiled product.
template <Weights W, bool MANY, bool LO, Read READ>
constexpr int kProductLds = MANY && !windowed(READ) ? std::max(kStretches<W, MANY, READ>, TiledProduct<W, 4, LO, READ>::kBytes)
                                                    : kStretches<W, MANY, READ>;

template <Weights W, bool MANY, Read READ>
__global__ __launch_bounds__((Shape<W, MANY>::kThreads), (Shape<W, MANY>::template kWavesPerSimd<READ>)) void gate_up_kernel(
    ExpertArgs a)
{
    typedef Shape<W, MANY> Sh;
    __shared__ __attribute__((aligned(16))) char lds[kProductLds<W, MANY, false, READ>];
    __shared__ float scales[Sh::kWaves * kScaleFloats<W, 2>];
    const Entry en(a.plan, blockIdx.y);
    [[maybe_unused]] const int z = blockIdx.z, nz = gridDim.z;  // of the workgroups that share an expert's tiles of tokens
    if constexpr (!MANY) {
        for (int r0 = 0; r0 < en.n; r0 += kTile)
            gate_up_stream<W, 1, Sh, READ>(a, en, r0, lds, scales);
    } else if (windowed(READ) || !a.tiled || en.n <= 2 * kTile) {
        for (int r0 = 2 * kTile * z; r0 < en.n; r0 += 2 * kTile * nz) {
            if (en.n - r0 <= kTile)
                gate_up_stream<W, 1, Sh, READ>(a, en, r0, lds, scales);
            else
                gate_up_stream<W, 2, Sh, READ>(a, en, r0, lds, scales);
        }
    } else if (static_cast<int>(blockIdx.x) * 4 * kTile < a.I) {
        if constexpr (!windowed(READ))
            for (int r0 = 4 * kTile * z; r0 < en.n; r0 += 4 * kTile * nz)
                gate_up_tiles<W, 4, READ>(a, en, r0, lds, scales);
    }
}

// ---------------------------------------------------------------- down product
// As the gate and up products, 32 rows of w_down (columns of out) to a unit, so that the two rows of h are read once
// for twice the weights. Each slot's product goes to a float32 row of its own; the merge adds them up. Where fewer than
// 32 columns are left a unit's second tile begins earlier, and both store the same values there. Memory bounds it, less
// well fed than the gate and up products by its shorter rows and twice the activations: the cases above 260 us, 5.4 TB/s; 45
// us, 4.4; 75 us, 3.0.
__device__ __forceinline__ int second_tile(const ExpertArgs &a, int c0)
{
    return min(kTile, max(a.H - kTile - c0, 0));
}

template <Weights W, Read READ>
__device__ __forceinline__ void down_weights(const ExpertArgs &a, const Entry &en, int unit, char *window, float *scales,
                                             WeightRows<W, 2, READ> &rows)
{
    const int c0 = min(unit * 2 * kTile, a.H - 1), c1 = second_tile(a, c0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = en.ex * a.H + c0 + i * c1;
        rows.w[i] = static_cast<const char *>(a.w) + row * a.I * sizeof(typename WeightType<W>::type);
        rows.scales.row[i] = a.scales + row * a.nb;
    }
    rows.rows_of(a.I, a.H - 1 - c0 - c1, window);
    rows.scales_of(a, a.H - 1 - c0 - c1, scales);
}

__device__ __forceinline__ void store_y(const ExpertArgs &a, const Entry &en, int row, int unit, int column, float first,
                                        float second)
{
    const int c0 = unit * 2 * kTile;
    if (row >= en.n || c0 >= a.H)
        return;
    float *y = a.y + static_cast<int64_t>(en.p0 + row) * a.H;
    const int c1 = second_tile(a, c0);
    if (c0 + column < a.H)
        y[c0 + column] = first;
    if (c1 > 0 && c0 + c1 + column < a.H)
        y[c0 + c1 + column] = second;
}

template <Weights W>
constexpr int kHRows = W == kWF32 ? 1 : 2;  // of h per slot

template <Weights W>
__device__ __forceinline__ const char *h_from(const ExpertArgs &a, int pos)
{
    return static_cast<const char *>(a.h) + static_cast<int64_t>(pos) * kHRows<W> * a.hI * sizeof(typename ActType<W>::type);
}

template <Weights W, int NT, typename Sh, Read READ>
__device__ __forceinline__ void down_stream(const ExpertArgs &a, const Entry &en, int r0, char *lds, float *scales)
{
    typedef typename ActType<W>::type X;
    Product<W, 2, NT, W != kWF32, Sh::kRegs, READ> p;
    const Share my(Sh::kWaves, a.parts);
    down_weights<W, READ>(a, en, my.unit, lds + wave_id() * Sh::template kStretch<READ>, scales, p.rows);
    p.lo = static_cast<int64_t>(a.hI) * sizeof(X);
    p.x = h_from<W>(a, en.p0 + r0);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = min(t * kTile + static_cast<int>(threadIdx.x % kTile), en.n - 1 - r0);
        p.x_row[t] = static_cast<uint32_t>(r * kHRows<W> * a.hI) * sizeof(X);
    }
    const int loads = (a.I + kLoadElems<W> - 1) / kLoadElems<W>;
    p.run(loads * my.part / a.parts, loads * (my.part + 1) / a.parts, a.I, a.stagger ? my.unit : 0);
    join_parts<Sh::kWaves, NT, Sh::template kStretch<READ>>(p.acc, a.parts, lds,
                                                            [&](int unit, int row, int column, const float (&v)[2]) {
        store_y(a, en, r0 + row, blockIdx.x * (Sh::kWaves / a.parts) + unit, column, v[0], v[1]);
    });
}

template <Weights W, int NT, Read READ>
__device__ __forceinline__ void down_tiles(const ExpertArgs &a, const Entry &en, int r0, char *lds, float *scales)
{
    typedef typename ActType<W>::type X;
    TiledProduct<W, NT, W != kWF32, READ> p;
    const int unit = blockIdx.x * 4 + wave_id(), lane = threadIdx.x & (kWave - 1);
    down_weights<W, READ>(a, en, unit, nullptr, scales, p.rows);
    p.lo = static_cast<int64_t>(a.hI) * sizeof(X);
    p.x = h_from<W>(a, en.p0 + r0);
    p.run(a.I, reinterpret_cast<u32x4 *>(lds), [&](int r) {
        return static_cast<uint32_t>(min(r, en.n - 1 - r0) * kHRows<W> * a.hI) * static_cast<uint32_t>(sizeof(X));
    });
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            store_y(a, en, r0 + t * kTile + lane / kTile * 4 + r, unit, lane % kTile, p.acc[0][t][r], p.acc[1][t][r]);
}

template <Weights W, bool MANY, Read READ>
__global__ __launch_bounds__((Shape<W, MANY>::kThreads), (Shape<W, MANY>::template kWavesPerSimd<READ>)) void down_kernel(
    ExpertArgs a)
{
    typedef Shape<W, MANY> Sh;
    __shared__ __attribute__((aligned(16))) char lds[kProductLds<W, MANY, W != kWF32, READ>];
    __shared__ float scales[Sh::kWaves * kScaleFloats<W, 2>];
    const Entry en(a.plan, blockIdx.y);
    [[maybe_unused]] const int z = blockIdx.z, nz = gridDim.z;  // of the workgroups that share an expert's tiles of tokens
    if constexpr (!MANY) {
        for (int r0 = 0; r0 < en.n; r0 += kTile)
            down_stream<W, 1, Sh, READ>(a, en, r0, lds, scales);
    } else if (windowed(READ) || !a.tiled || en.n <= kTile) {
        for (int r0 = 2 * kTile * z; r0 < en.n; r0 += 2 * kTile * nz) {
            if (en.n - r0 <= kTile)
                down_stream<W, 1, Sh, READ>(a, en, r0, lds, scales);
            else
                down_stream<W, 2, Sh, READ>(a, en, r0, lds, scales);
        }
    } else if (static_cast<int>(blockIdx.x) * 4 * 2 * kTile < a.H) {
        if constexpr (!windowed(READ))
            for (int r0 = 4 * kTile * z; r0 < en.n; r0 += 4 * kTile * nz) {
                if (en.n - r0 <= 2 * kTile)
                    down_tiles<W, 2, READ>(a, en, r0, lds, scales);
                else
                    down_tiles<W, 4, READ>(a, en, r0, lds, scales);
            }
    }
}

// ---------------------------------------------------------------- down product with the merge
// For up to 16 tokens and little to read: one workgroup per 16 columns of out and all experts in use, whose wavefronts
// share the (expert, load) pairs in order, each a stretch. A wavefront adds its tiles into sums of its own, [T][16] in
// LDS, when its expert changes; the wavefronts' sums are put together in order.
constexpr int kDirectThreads = 1024, kDirectWaves = kDirectThreads / kWave;

__device__ __forceinline__ void store_out(const ExpertArgs &a, int t, int c, float v)
{
    const int64_t o = static_cast<int64_t>(t) * a.H + c;
    if (a.out_bf16) {
        if (a.bias)
            v += to_f32(static_cast<const uint16_t *>(a.bias)[o]);
        static_cast<uint16_t *>(a.out)[o] = static_cast<uint16_t>(f32_to_bf16_bits(v));
    } else {
        if (a.bias)
            v += static_cast<const float *>(a.bias)[o];
        static_cast<float *>(a.out)[o] = v;
    }
}

template <Weights W, Read READ>
__global__ __launch_bounds__(kDirectThreads) void down_merge_kernel(ExpertArgs a)
{
    typedef Product<W, 1, 1, W != kWF32, Shape<W, false>::kRegs, READ> P;
    __shared__ float sums[kDirectWaves][kTile][kTile], scales[kDirectWaves * kScaleFloats<W, 1>];
    const int lane = threadIdx.x & (kWave - 1), wave = wave_id(), m = lane % kTile, g = lane / kTile;
    const int c0 = blockIdx.x * kTile;
    for (int i = lane; i < kTile * kTile; i += kWave)
        sums[wave][i / kTile][i % kTile] = 0.0f;
    const int loads = (a.I + kLoadElems<W> - 1) / kLoadElems<W>, all = a.plan.head[0] * loads;
    const int u1 = all * (wave + 1) / kDirectWaves;
    for (int u = all * wave / kDirectWaves; u < u1;) {
        const int i = u / loads, l0 = u - i * loads, l1 = min(loads, l0 + (u1 - u));
        u += l1 - l0;
        const int p0 = a.plan.start[i], n = a.plan.start[i + 1] - p0;
        const int64_t row = static_cast<int64_t>(a.plan.act[i]) * a.H + c0;
        for (int r0 = 0; r0 < n; r0 += kTile) {
            P p;
            p.rows.w[0] = static_cast<const char *>(a.w) + row * a.I * sizeof(typename P::Wt);
            p.rows.scales.row[0] = a.scales + row * a.nb;
            p.rows.rows_of(a.I, a.H - 1 - c0, nullptr);
            p.rows.scales_of(a, a.H - 1 - c0, scales);
            p.lo = static_cast<int64_t>(a.hI) * sizeof(typename P::X);
            p.x = h_from<W>(a, p0 + r0);
            const int r = min(m, n - 1 - r0), tok = a.plan.token[p0 + r0 + r];
            p.x_row[0] = static_cast<uint32_t>(r * kHRows<W> * a.hI) * sizeof(typename P::X);
            p.run(l0, l1, a.I, 0);
            // this lane holds column m of the tile's rows 4 g .. 4 g + 3. A token that names the expert twice has two
            // rows, neighbours: then the lane groups add one after the other
            const bool twice = __ballot(m > 0 && r0 + m < n && tok == __shfl_up(tok, 1)) != 0;
            for (int turn = 0; turn < (twice ? 4 : 1); ++turn) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int to = __shfl(tok, 4 * g + q);
                    if ((!twice || g == turn) && r0 + 4 * g + q < n)
                        sums[wave][to][m] += p.acc[0][0][q];
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
    }
    __syncthreads();
    const int t = threadIdx.x / kTile, c = c0 + threadIdx.x % kTile;
    if (t >= a.T || c >= a.H)
        return;
    float v = 0.0f;
    for (int k = 0; k < kDirectWaves; ++k)
        v += sums[k][t][threadIdx.x % kTile];
    store_out(a, t, c, v);
}

// ---------------------------------------------------------------- merge
// out[t] = the sum of its slots' rows in slot order (their weights are in h), plus bias. Little more than a launch: 4.5 us at
// T1 H7168 K8, 5.1 at T64.
constexpr int kMergeThreads = 256;

__global__ __launch_bounds__(kMergeThreads) void merge_kernel(ExpertArgs a)
{
    const int c = blockIdx.x * kMergeThreads + threadIdx.x, t = blockIdx.y;
    if (c >= a.H)
        return;
    float v = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += 8) {  // eight slots' loads in flight together
        int pos[8];
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            pos[k] = k0 + k < a.K ? a.plan.place[t * a.K + k0 + k] : -1;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = a.y[static_cast<int64_t>(max(pos[k], 0)) * a.H + c];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v += pos[k] >= 0 ? y[k] : 0.0f;
    }
    store_out(a, t, c, v);
}

// ---------------------------------------------------------------- host side
// I rounded up to whole lines of bf16: the stride of h's rows (all of them begin on a line of the workspace's alignment).
int64_t line_elems(int64_t I) { return (I + 63) & ~int64_t{63}; }

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// The workspace: parts of the logits, logits, plan, h.
struct Layout {
    size_t part, logits, head, act, start, order, token, place, h, y, bytes;
};

Layout layout(int64_t T, int64_t H, int64_t E, int64_t K, int64_t I)
{
    Layout l{};
    const int64_t slots = T * K, used = E < slots ? E : slots;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += round16(n);
        return here;
    };
    l.part = take(8 * router_splits(T, E, H) * T * E);
    l.logits = take(4 * T * E);
    l.head = take(4);
    l.act = take(4 * used);
    l.start = take(4 * (used + 1));
    l.order = take(4 * slots);
    l.token = take(4 * slots);
    l.place = take(4 * slots);
    l.h = take(4 * slots * line_elems(I));
    l.y = take(4 * slots * H);
    l.bytes = at;
    return l;
}

// The layer's own routing names K different experts (`distinct`); a routing that the caller has may name fewer of them, or one
// several times, and then E, the experts held here, may be less than K.
moe_status check_sizes(int64_t T, int64_t H, int64_t I, int32_t E, int32_t K, bool distinct)
{
    if (T < 0 || H < 1 || I < 1 || E < 1 || K < 1 || (distinct && K > E))
        return MOE_ERR_INVALID;
    if (T > kMaxFewTokens || E > MOE_MAX_EXPERTS || K > MOE_MAX_TOPK || H > (1 << 20) || I > (1 << 20))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t K, bool distinct, size_t *bytes)
{
    if (!bytes)
        return MOE_ERR_INVALID;
    const moe_status st = check_sizes(T, H, I, E, K, distinct);
    if (st != MOE_OK)
        return st;
    *bytes = T == 0 ? 0 : layout(T, H, E, K, I).bytes;
    return MOE_OK;
}

Plan plan_in(char *ws, const Layout &l)
{
    return Plan{reinterpret_cast<int32_t *>(ws + l.head), reinterpret_cast<int32_t *>(ws + l.act),
                reinterpret_cast<int32_t *>(ws + l.start), reinterpret_cast<int32_t *>(ws + l.order),
                reinterpret_cast<int32_t *>(ws + l.token), reinterpret_cast<int32_t *>(ws + l.place)};
}

struct ExpertWeights {
    const void *gate_up, *down;
    moe_dtype dt;
    const float *gate_up_scales, *down_scales;
    int32_t block;
};

moe_status check_layer(const void *x, moe_dtype dt, int64_t T, int64_t H, int64_t I, int32_t E, int32_t K,
                       const ExpertWeights &w, const void *out, moe_dtype out_dt, const void *workspace,
                       size_t workspace_bytes, bool distinct)
{
    const moe_status st = check_sizes(T, H, I, E, K, distinct);
    if (st != MOE_OK)
        return st;
    if ((dt != MOE_F32 && dt != MOE_BF16 && dt != MOE_FP8_E4M3) || (w.dt != MOE_F32 && w.dt != MOE_BF16 && w.dt != MOE_FP8_E4M3) ||
        (out_dt != MOE_F32 && out_dt != MOE_BF16 && out_dt != MOE_FP8_E4M3))
        return MOE_ERR_INVALID;
    if (dt == MOE_FP8_E4M3 || out_dt == MOE_FP8_E4M3 || (w.dt != dt && !(dt == MOE_BF16 && w.dt == MOE_FP8_E4M3)))
        return MOE_ERR_UNSUPPORTED;
    if (w.dt == MOE_FP8_E4M3) {
        if (w.block < 1 || H % w.block || I % w.block)
            return MOE_ERR_INVALID;
        if (w.block % kLoadElems<kWFp8>)
            return MOE_ERR_UNSUPPORTED;
    }
    if (T == 0)
        return MOE_OK;
    if (!x || !w.gate_up || !w.down || !out || (w.dt == MOE_FP8_E4M3 && (!w.gate_up_scales || !w.down_scales)))
        return MOE_ERR_INVALID;
    if (!workspace || !aligned16(workspace) || workspace_bytes < layout(T, H, E, K, I).bytes)
        return MOE_ERR_INVALID;
    return MOE_OK;
}

// Bytes of router weights up to which one workgroup reads them all and routes too.
constexpr int64_t kSmallRouter = 128 << 10;

size_t plan_lds(int E) { return sizeof(uint16_t) * kPlanWaves * static_cast<size_t>(E); }

// The host does not know how many experts a call uses: `used` of the rules below is the most there may be, min(E, T K), and so
// are the sizes beside them (routers whose logits have something in common use a third to two thirds of them).

// Wavefronts that share a unit of weight rows: more of them while the chip has not several rounds of wavefronts (T8 H4096
// I2048 E128 K8 FP8 with four against two: 189 -> 181 us and 112 -> 106; T64 H7168 I1024 E128 K8 down, 28672 units, with four
// against one: 333 -> 388), as long as each keeps four loads or more (T32 H1024 I512 E64 K4 down with two: 23 -> 32 us).
// Through the window each of them reads a line more, so they are fewer (T133 H2056 I1399 E64 K2 with the others' limits 292
// us, with 16 loads 256, with 8192 units too 234).
int share_parts(int64_t units, int64_t loads, int waves, bool window)
{
    int parts = 1;
    while (parts < waves && units * parts < (window ? 8192 : 24576) && loads >= (window ? 16 : 8) * parts)
        parts *= 2;
    return parts;
}

// Rows a multiple of 4 KiB apart begin on the same memory channels, and wavefronts that run side by side would ask them
// for the same columns at the same time: there each begins with another load (T64 H4096 I2048 E64 K2: gate and up 352 ->
// 329 us, down 187 -> 161; rows of 2 or 14 KiB are up to 7% faster read from the start).
bool stagger(int64_t row_bytes) { return row_bytes % 4096 == 0; }

// Loads of a column tile's experts (by the most experts that may be in use) up to which one workgroup takes them all and
// merges too: a launch fewer, which is what the smallest calls spend their time on (T1 H512 I1024 K2 float32 21 -> 19 us),
// against less of the chip at work (T8 H1024 I512 K4, 112 loads: 21 -> 32 us). In between, replayed from a graph: 64 loads 24
// and 24 us, 70 25 -> 24, 80 26 -> 27, 96 24 -> 28, 29 -> 30 and 35 -> 38.
constexpr int64_t kDirectLoads = 64;

// Workgroups from which on the tiled product, whose wavefronts do not share a unit's loads, has the chip filled: T256 H4096
// I2048 E16 K4 with 512 of them 290 -> 219 us (gate and up); T100 H4096 I1024 E8 K2 with 128 44 -> 88, down with 256 35 ->
// 43. Gate and up take it from 33 tokens an expert, down, whose activations are twice the bytes, from 17 (T200 H7168 I1024
// E64 K8, 25 tokens an expert: 446 -> 568 us and 335 -> 290).
constexpr int64_t kTiledGroups = 512;

// Rows off the cache lines go through the window where there is much to read (kWindowWork loads of all units, 100 MB) for
// few tokens an expert: a wavefront's stretch costs a line more that way, and a step through LDS, which the tiled product
// and small calls do not earn back (T133 H2056 I1399 E64 K2 304 -> 234 us, T64 H7170 I1026 E64 K8 700 -> 564, T8 H2057 I1399
// E64 K4 float32 197 -> 177; with the window T4 H1000 I500 E16 K4 22 -> 42, T200 H4100 I2050 E16 K4 309 -> 354).
constexpr int64_t kWindowWork = 24576;

template <Weights W>
Read read_of(const void *w, int64_t row_bytes, const void *x, int64_t x_row_bytes, bool window)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(w) | static_cast<uintptr_t>(row_bytes);
    const bool odd_x = W == kWBf16 && (reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(x_row_bytes)) % 4;
    if (at % 128 == 0 && !odd_x)
        return kLines;
    if (window)
        return odd_x ? kWindowOdd : kWindow;
    return odd_x || (W == kWBf16 && at % 4) ? kOdd : kWords;
}

// Workgroups that take an expert's tiles of tokens in turn, where there may be several: an expert with many tokens among others
// with few would be what a call ends with. They are the slowest index of the grid, so that all experts' first tiles begin
// before any second ones, and two of an expert share no read of its weights. T133 H2056 I1399 E64 K2 with experts of 1 to 55
// tokens 192 -> 174 us; T256 H4096 I2048 E16 K4 FP8 230 -> 215; with four of them 172 and 215, but T64 H4096 I2048 E64 K4 FP8
// 332 -> 343.
unsigned turns(int T) { return T > 2 * kTile ? 2u : 1u; }

template <Weights W, bool MANY>
void launch_products(ExpertArgs a, const ExpertWeights &w, int used, hipStream_t stream)
{
    typedef Shape<W, MANY> Sh;
    constexpr int size = sizeof(typename WeightType<W>::type);
    // FP8: the scale of load l is l / (loads per block), by a multiplication (exact for l * block / 128 < 2^32)
    const int lb = W == kWFp8 ? w.block / kLoadElems<kWFp8> : 1;
    a.per_block = lb == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + lb - 1) / lb);
    a.w = w.gate_up;
    a.scales = w.gate_up_scales;
    a.nb = W == kWFp8 ? a.H / w.block : 0;
    a.stagger = stagger(int64_t{a.H} * size);
    int64_t units = ceil_div(a.I, kTile);
    a.tiled = MANY && units / 4 * used >= kTiledGroups;
    int64_t loads = ceil_div(a.H, kLoadElems<W>);
    const bool few = a.T * a.K <= kTile * used;
    Read read = read_of<W>(a.w, int64_t{a.H} * size, a.x, int64_t{a.H} * sizeof(typename ActType<W>::type),
                           (few || !a.tiled) && units * used * loads >= kWindowWork);
    a.parts = share_parts(units * used, loads, Sh::kWaves, windowed(read));
    dim3 grid(static_cast<unsigned>(ceil_div(units, Sh::kWaves / a.parts)), static_cast<unsigned>(used), MANY ? turns(a.T) : 1u);
#define MOE_FEW_PRODUCT(KERNEL, READ) hipLaunchKernelGGL((KERNEL<W, MANY, READ>), grid, dim3(Sh::kThreads), 0, stream, a)
    if (read == kLines)
        MOE_FEW_PRODUCT(gate_up_kernel, kLines);
    else if (read == kWindow)
        MOE_FEW_PRODUCT(gate_up_kernel, kWindow);
    else if (W != kWBf16 || read == kWords)
        MOE_FEW_PRODUCT(gate_up_kernel, kWords);
    else if constexpr (W == kWBf16) {
        if (read == kOdd)
            MOE_FEW_PRODUCT(gate_up_kernel, kOdd);
        else
            MOE_FEW_PRODUCT(gate_up_kernel, kWindowOdd);
    }
    a.w = w.down;
    a.scales = w.down_scales;
    a.nb = W == kWFp8 ? a.I / w.block : 0;
    a.stagger = stagger(int64_t{a.I} * size);
    units = ceil_div(a.H, 2 * kTile);
    a.tiled = MANY && units / 4 * used >= kTiledGroups;
    loads = ceil_div(a.I, kLoadElems<W>);
    if (!MANY && used * loads <= kDirectLoads) {
        read = read_of<W>(a.w, int64_t{a.I} * size, nullptr, 0, false);
        grid = dim3(static_cast<unsigned>(ceil_div(a.H, kTile)));
        if (read == kLines)
            hipLaunchKernelGGL((down_merge_kernel<W, kLines>), grid, dim3(kDirectThreads), 0, stream, a);
        else if (W != kWBf16 || read == kWords)
            hipLaunchKernelGGL((down_merge_kernel<W, kWords>), grid, dim3(kDirectThreads), 0, stream, a);
        else if constexpr (W == kWBf16)
            hipLaunchKernelGGL((down_merge_kernel<W, kOdd>), grid, dim3(kDirectThreads), 0, stream, a);
        return;
    }
    read = read_of<W>(a.w, int64_t{a.I} * size, nullptr, 0, (few || !a.tiled) && units * used * loads >= kWindowWork);
    a.parts = share_parts(units * used, loads, Sh::kWaves, windowed(read));
    grid = dim3(static_cast<unsigned>(ceil_div(units, Sh::kWaves / a.parts)), static_cast<unsigned>(used), MANY ? turns(a.T) : 1u);
    if (read == kLines)
        MOE_FEW_PRODUCT(down_kernel, kLines);
    else if (read == kWindow)
        MOE_FEW_PRODUCT(down_kernel, kWindow);
    else if (W != kWBf16 || read == kWords)
        MOE_FEW_PRODUCT(down_kernel, kWords);
    else if constexpr (W == kWBf16)
        MOE_FEW_PRODUCT(down_kernel, kOdd);
#undef MOE_FEW_PRODUCT
    hipLaunchKernelGGL(merge_kernel, dim3(static_cast<unsigned>(ceil_div(a.H, kMergeThreads)), static_cast<unsigned>(a.T)),
                       dim3(kMergeThreads), 0, stream, a);
}

template <Weights W>
void launch_products_of(const ExpertArgs &a, const ExpertWeights &w, int used, hipStream_t stream)
{
    if (a.T <= kTile)
        launch_products<W, false>(a, w, used, stream);
    else
        launch_products<W, true>(a, w, used, stream);
}

moe_status launch_experts(const void *x, int64_t T, int64_t H, int64_t I, int32_t E, int32_t K, const int32_t *topk_idx,
                          const float *topk_w, const ExpertWeights &w, const void *bias, void *out, moe_dtype out_dt,
                          char *ws, bool planned, hipStream_t stream)
{
    const Layout l = layout(T, H, E, K, I);
    const int slots = static_cast<int>(T * K), used = E < slots ? E : slots;
    ExpertArgs a{};
    a.plan = plan_in(ws, l);
    a.x = x;
    a.topk_w = topk_w;
    a.h = ws + l.h;
    a.y = reinterpret_cast<float *>(ws + l.y);
    a.bias = bias;
    a.out = out;
    a.out_bf16 = out_dt == MOE_BF16;
    a.T = static_cast<int>(T);
    a.K = K;
    a.H = static_cast<int>(H);
    a.I = static_cast<int>(I);
    a.hI = static_cast<int>(line_elems(I));
    if (!planned)
        hipLaunchKernelGGL(few_token_plan_kernel, dim3(1), dim3(kPlanThreads), plan_lds(E), stream, topk_idx, slots, E, K,
                           a.plan);
    if (w.dt == MOE_FP8_E4M3)
        launch_products_of<kWFp8>(a, w, used, stream);
    else if (w.dt == MOE_F32)
        launch_products_of<kWF32>(a, w, used, stream);
    else
        launch_products_of<kWBf16>(a, w, used, stream);
    return launch_status();
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_few_token_workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t K, size_t *bytes)
{
    return moe::workspace_size(T, H, I, E, K, true, bytes);
}

extern "C" moe_status moe_few_token_experts_workspace_size(int64_t T, int64_t H, int64_t I, int32_t E, int32_t K,
                                                           size_t *bytes)
{
    return moe::workspace_size(T, H, I, E, K, false, bytes);
}

extern "C" moe_status moe_few_token_experts(const void *x, moe_dtype dt, int64_t T, int64_t H, int64_t I, int32_t E,
                                            int32_t K, const int32_t *topk_idx, const float *topk_w,
                                            const void *w_gate_up, const void *w_down, moe_dtype weight_dt,
                                            const float *gate_up_scales, const float *down_scales, int32_t block,
                                            const void *bias, void *out, moe_dtype out_dt, void *workspace,
                                            size_t workspace_bytes, hipStream_t stream)
{
    using namespace moe;
    const ExpertWeights w{w_gate_up, w_down, weight_dt, gate_up_scales, down_scales, block};
    const moe_status st = check_layer(x, dt, T, H, I, E, K, w, out, out_dt, workspace, workspace_bytes, false);
    if (st != MOE_OK || T == 0)
        return st;
    if (!topk_idx)
        return MOE_ERR_INVALID;
    return launch_experts(x, T, H, I, E, K, topk_idx, topk_w, w, bias, out, out_dt, static_cast<char *>(workspace),
                          false, stream);
}

extern "C" moe_status moe_few_token_layer(const void *x, moe_dtype dt, const void *router, int64_t T, int64_t H,
                                          int64_t I, int32_t E, int32_t K, int32_t route_group_size,
                                          int32_t topk_groups, const void *w_gate_up, const void *w_down,
                                          moe_dtype weight_dt, const float *gate_up_scales, const float *down_scales,
                                          int32_t block, const void *bias, void *out, moe_dtype out_dt,
                                          int32_t *topk_idx, float *topk_w, void *workspace, size_t workspace_bytes,
                                          hipStream_t stream)
{
    using namespace moe;
    const ExpertWeights w{w_gate_up, w_down, weight_dt, gate_up_scales, down_scales, block};
    moe_status st = check_layer(x, dt, T, H, I, E, K, w, out, out_dt, workspace, workspace_bytes, true);
    if (st != MOE_OK)
        return st;
    // the routing's own argument errors, before anything is launched
    const int32_t gs = route_group_size > 0 ? route_group_size : 0;
    st = gs ? moe_route_topk_grouped(nullptr, 0, E, K, gs, topk_groups, nullptr, nullptr, stream) : MOE_OK;
    if (st != MOE_OK || T == 0)
        return st;
    if (!router || !topk_idx || !topk_w)
        return MOE_ERR_INVALID;
    char *ws = static_cast<char *>(workspace);
    const Layout l = layout(T, H, E, K, I);
    double *part = reinterpret_cast<double *>(ws + l.part);
    const int Ti = static_cast<int>(T), Hi = static_cast<int>(H), splits = router_splits(T, E, H);
    if (gs == 0 && T <= kTile && E <= kSmallExperts && E * H * (dt == MOE_F32 ? 4 : 2) <= kSmallRouter) {
        const Plan plan = plan_in(ws, l);
        if (dt == MOE_F32)
            hipLaunchKernelGGL(few_token_small_route_kernel<float>, dim3(1), dim3(kPlanThreads), plan_lds(E), stream,
                               static_cast<const float *>(x), static_cast<const float *>(router), Ti, Hi, E, K, topk_idx,
                               topk_w, plan);
        else
            hipLaunchKernelGGL(few_token_small_route_kernel<uint16_t>, dim3(1), dim3(kPlanThreads), plan_lds(E), stream,
                               static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(router), Ti, Hi, E, K, topk_idx,
                               topk_w, plan);
        return launch_experts(x, T, H, I, E, K, topk_idx, topk_w, w, bias, out, out_dt, ws, true, stream);
    }
    const dim3 grid(static_cast<unsigned>(ceil_div(E, kTile)), static_cast<unsigned>(ceil_div(T, kTile)),
                    static_cast<unsigned>(splits));
    if (dt == MOE_F32)
        hipLaunchKernelGGL(router_kernel<float>, grid, dim3(kRouterThreads), 0, stream, static_cast<const float *>(x),
                           static_cast<const float *>(router), Ti, Hi, E, part);
    else
        hipLaunchKernelGGL(router_kernel<uint16_t>, grid, dim3(kRouterThreads), 0, stream, static_cast<const uint16_t *>(x),
                           static_cast<const uint16_t *>(router), Ti, Hi, E, part);
    const bool planned = gs == 0 && T <= kPlanWaves;
    if (gs) {
        float *logits = reinterpret_cast<float *>(ws + l.logits);
        hipLaunchKernelGGL(router_sum_kernel, dim3(static_cast<unsigned>(ceil_div(T * E, kRouterThreads))),
                           dim3(kRouterThreads), 0, stream, part, splits, Ti * E, logits);
        st = moe_route_topk_grouped(logits, T, E, K, gs, topk_groups, topk_idx, topk_w, stream);
        if (st != MOE_OK)
            return st;
    } else {
        const Plan plan = plan_in(ws, l);
#define MOE_FEW_ROUTE(J, PLAN)                                                                                       \
    hipLaunchKernelGGL((few_token_route_kernel<J, PLAN>), dim3(static_cast<unsigned>(ceil_div(T, kPlanWaves))),        \
                       dim3(kPlanThreads), PLAN ? plan_lds(E) : 0, stream, part, splits, Ti, E, K, topk_idx, topk_w, plan)
        if (E <= 4 * kWave) {
            if (planned)
                MOE_FEW_ROUTE(4, true);
            else
                MOE_FEW_ROUTE(4, false);
        } else {
            if (planned)
                MOE_FEW_ROUTE(16, true);
            else
                MOE_FEW_ROUTE(16, false);
        }
#undef MOE_FEW_ROUTE
    }
    return launch_experts(x, T, H, I, E, K, topk_idx, topk_w, w, bias, out, out_dt, ws, planned, stream);
}
