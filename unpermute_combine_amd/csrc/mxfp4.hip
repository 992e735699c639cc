// Rows in microscaled 4-bit floating point (OCP MX: E2M1 codes, one E8M0 scale for each 32 consecutive elements of a row),
// and the products of the experts' rows with their weights in that form.
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

// Eight consecutive elements, at any address of their type.
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8])
{
    u32x4 q;
    __builtin_memcpy(&q, p, sizeof(q));
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    __builtin_memcpy(v, p, sizeof(v));
}

// Four lanes a block, eight elements a lane. Rows are whole blocks, so the tensor is one run of them.
template <typename X>
__global__ __launch_bounds__(kMxThreads) void quantize_mxfp4_kernel(const X *__restrict__ x, int64_t blocks,
                                                                    uint8_t *__restrict__ q, uint8_t *__restrict__ scales)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kMxThreads + threadIdx.x;  // eight elements
    if (i / 4 >= blocks)
        return;
    float v[8];
    load8(x + 8 * i, v);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    top = max_dpp<kDppQuadXor2>(max_dpp<kDppQuadXor1>(top));
    const int32_t biased = static_cast<int32_t>(top >> 23);  // floor(log2 amax) + 127, or less than -126 as 0
    const uint32_t byte = biased == 255 ? kMxNan : top == 0 ? 127u : static_cast<uint32_t>(max(biased - 2, 0));
    // the conversion takes the scale as a float32 whose exponent field counts (0: 2^-127)
    const float scale = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
    uint32_t w = 0;
    if (byte != kMxNan) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
    }
    __builtin_memcpy(q + 4 * i, &w, sizeof(w));
    if (i % 4 == 0)
        scales[i / 4] = static_cast<uint8_t>(byte);
}

template <typename X>
moe_status launch_quantize(const void *x, int64_t blocks, uint8_t *q, uint8_t *scales, hipStream_t stream)
{
    const int64_t grid = ceil_div(4 * blocks, kMxThreads);
    if (grid > 0x7fffffff)
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
