// w4a4_epilogue.h -- pieces of the W4A4 linears' epilogues shared by the tile
// kernels (w4a4_gemm.hip) and the few-row kernel (w4a4_few.hip).
#pragma once

#include "svdq_internal.h"
#include "svdq_quant.h"

namespace svdq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_to_f32(uint32_t b) { return bits_f32(b << 16); }

// two fp32 -> two bf16 (round to nearest even), packed low | high << 16
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// GELU, tanh form: 0.5 y (1 + tanh(u)) = y / (1 + exp(-2u)),
// u = sqrt(2/pi) (y + 0.044715 y^3); exp via the hardware exp2.
__device__ __forceinline__ float gelu_tanh(float y)
{
    const float k1 = -2.302208198f;      // -2 sqrt(2/pi) log2(e)
    const float k3 = -0.102943836f;      // -2 sqrt(2/pi) 0.044715 log2(e)
    const float t = y * __builtin_fmaf(k3, y * y, k1);
    return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}

// SiLU: y / (1 + exp(-y)).
__device__ __forceinline__ float silu(float y)
{
    return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * y));
}

// 8 fp32 values of h -> bf16 hi and lo parts (hi = bf16(h), lo = bf16(h - hi)).
__device__ __forceinline__ void split_h(const float *hv, bf16x8 &hi8, bf16x8 &lo8)
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = pack_bf16x2(hv[2 * i], hv[2 * i + 1]);
        lo[i] = pack_bf16x2(hv[2 * i] - bf16_to_f32(hi[i] & 0xFFFFu), hv[2 * i + 1] - bf16_to_f32(hi[i] >> 16));
    }
    hi8 = __builtin_bit_cast(bf16x8, (uint4){hi[0], hi[1], hi[2], hi[3]});
    lo8 = __builtin_bit_cast(bf16x8, (uint4){lo[0], lo[1], lo[2], lo[3]});
}

__device__ __forceinline__ void load_h8(const float *__restrict__ h, int m, int M, int k, float *hv)
{
    if (m < M) {
        const float4 a = *reinterpret_cast<const float4 *>(h + (size_t)m * 32 + k);
        const float4 b = *reinterpret_cast<const float4 *>(h + (size_t)m * 32 + k + 4);
        hv[0] = a.x; hv[1] = a.y; hv[2] = a.z; hv[3] = a.w;
        hv[4] = b.x; hv[5] = b.y; hv[6] = b.z; hv[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) hv[i] = 0.0f;
    }
}

}  // namespace
}  // namespace svdq
