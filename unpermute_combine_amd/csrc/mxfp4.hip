// Rows in microscaled 4-bit floating point (OCP MX: E2M1 codes, one E8M0 scale for each 32 consecutive elements of a row).
//   amax = max |x|, scale = 2^(floor(log2 amax) - 2)  (6 = 1.5 * 2^2 is the largest code), byte = exponent + 127
//   code = E2M1 of x / scale, nearest, ties to the even code, 6 beyond it
#include <algorithm>

#include "moe_common.h"

namespace moe {
namespace {

constexpr int kMxBlock = 32;
constexpr int kMxThreads = 256;
constexpr uint32_t kMxNan = 255;  // the scale byte of a block that holds a NaN or an infinity

constexpr int kDppQuadXor2 = 0x4e;
constexpr int kDppQuadXor1 = 0xb1;

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v)
{
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false)));
}

// Eight consecutive elements, at any address of their type. bf16 rows are read past the caches, four vectors a thread: 46.0 us at
// T16384 H7168 (6.5 TB/s, a large read's rate) against 50.4 by one ordinary load a thread; where the rows are in the caches it
// costs a little (T8192 H4096 14.5 against 14.0). float32 rows, whose lanes take two vectors, gain nothing (T16384 H4096 52.2 us,
// 56 with four).
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8])
{
    typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
    const vec q = __builtin_nontemporal_load(reinterpret_cast<const vec *>(p));
    v[0] = bf16_lo(q[0]); v[1] = bf16_hi(q[0]); v[2] = bf16_lo(q[1]); v[3] = bf16_hi(q[1]);
    v[4] = bf16_lo(q[2]); v[5] = bf16_hi(q[2]); v[6] = bf16_lo(q[3]); v[7] = bf16_hi(q[3]);
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    __builtin_memcpy(v, p, sizeof(v));
}

template <typename X> constexpr int kEach = sizeof(X) == 2 ? 4 : 1;  // vectors of eight elements a thread

// Four lanes a block, eight elements a lane: the largest magnitude's bits by two DPP steps, the codes by the conversion instruction,
// which gives the definition's for every element and scale (tested). Rows are whole blocks, so the tensor is one run of them.
// Memory bound: T16384 H7168 bf16 297 MB in 46 us. Small calls are the host's (T8 H7168 2.7 us on the GPU).
template <typename X>
__global__ __launch_bounds__(kMxThreads) void quantize_mxfp4_kernel(const X *__restrict__ x, int64_t blocks,
                                                                    uint8_t *__restrict__ q, uint8_t *__restrict__ scales)
{
    constexpr int kN = kEach<X>;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kMxThreads * kN) + threadIdx.x;
    float v[kN][8];
#pragma unroll
    for (int u = 0; u < kN; ++u)
        load8(x + 8 * min(first + u * kMxThreads, 4 * blocks - 1), v[u]);
#pragma unroll
    for (int u = 0; u < kN; ++u) {
        const int64_t i = first + u * kMxThreads;
        if (i >= 4 * blocks)
            return;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, __float_as_uint(v[u][j]) & 0x7fffffffu);
        top = max_dpp<kDppQuadXor2>(max_dpp<kDppQuadXor1>(top));
        const int32_t biased = static_cast<int32_t>(top >> 23);  // floor(log2 amax) + 127, or less than -126 as 0
        const uint32_t byte = biased == 255 ? kMxNan : top == 0 ? 127u : static_cast<uint32_t>(max(biased - 2, 0));
        // the conversion takes the scale as a float32 whose exponent field counts (0: 2^-127)
        const float scale = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[u][0], v[u][1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[u][2], v[u][3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[u][4], v[u][5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[u][6], v[u][7], scale, 3);
        w = byte == kMxNan ? 0 : w;
        __builtin_memcpy(q + 4 * i, &w, sizeof(w));
        if (i % 4 == 0)
            scales[i / 4] = static_cast<uint8_t>(byte);
    }
}

template <typename X>
moe_status launch_quantize(const void *x, int64_t blocks, uint8_t *q, uint8_t *scales, hipStream_t stream)
{
    const int64_t grid = ceil_div(4 * blocks, kMxThreads * kEach<X>);
    if (grid > 0xffffffff / kMxThreads)  // a grid's threads are a 32-bit number
        return MOE_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((quantize_mxfp4_kernel<X>), dim3(static_cast<unsigned>(grid)), dim3(kMxThreads), 0, stream,
                       static_cast<const X *>(x), blocks, q, scales);
    return launch_status();
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_quantize_mxfp4(const void *x, moe_dtype x_dt, int64_t T, int64_t H, uint8_t *q, uint8_t *scales,
                                         hipStream_t stream)
{
    using namespace moe;
    if (T < 0 || H < 1 || H % kMxBlock != 0 || (x_dt != MOE_F32 && x_dt != MOE_BF16 && x_dt != MOE_FP8_E4M3))
        return MOE_ERR_INVALID;
    if (x_dt == MOE_FP8_E4M3 || T > 0x7fffffff || H > (int64_t{1} << 26))
        return MOE_ERR_UNSUPPORTED;
    if (T == 0)
        return MOE_OK;
    if (!x || !q || !scales)
        return MOE_ERR_INVALID;
    const int64_t blocks = T * (H / kMxBlock);
    return x_dt == MOE_F32 ? launch_quantize<float>(x, blocks, q, scales, stream)
                           : launch_quantize<uint16_t>(x, blocks, q, scales, stream);
}
