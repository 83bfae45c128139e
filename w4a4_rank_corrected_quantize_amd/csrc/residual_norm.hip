// residual_norm.hip -- the step between two 4-bit linears of a transformer
// block: norm of the block's output, gate and residual scale, norm of the new
// residual stream and its modulation, in one pass over the rows.
//
//   t  = post(y_m) * post_w                    post: none, RMS or LayerNorm
//   r' = r_m + (alpha gate_b) t                stored in the stream's type
//   x  = (pre(r') * pre_w + pre_b) (1 + scale_b) + shift_b        bf16
//   RMS(v) = v / sqrt(mean(v^2) + eps);  LayerNorm(v) = RMS(v - mean(v))
//
// Everything between the loads and the two stores is fp32: x is formed from
// the unrounded r' (one rounding each for r' and x).  The variance is taken
// of the centred values held in registers, not as a difference of moments.
//
// Bound by HBM: r and y are read once, r' and x written once; the modulation
// vectors are shared by many rows and come from the L2.  Rows of up to 1024
// channels take a wave each (no barrier), longer ones a block of four; a row
// stays in registers between its sums.  9216 x 4096 bf16, LayerNorm and
// modulation: 53 us in the kernel for 302 MB = 5.7 TB/s (a large copy: 5.4; the
// last-level cache keeps part of the buffers from pass to pass; with conditions
// on the loads: 61 us); fp32 stream, a norm on both sides: 88 us for 453 MB.  1337 x 2560, fp32 stream, a norm on
// both sides: 11 us = 3.7 TB/s, five rows per compute unit and two sums in turn.
// One row of 4096: 3 us, the launch and three dependent passes of sums.
#include "launch_grid.h"
#include "svdq_internal.h"
#include "svdq_quant.h"

namespace svdq {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t rn_pack2(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));   // round to nearest even
}

__device__ __forceinline__ void rn_unpack8(const uint4 &u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bits_f32(w[i] << 16);
        f[2 * i + 1] = bits_f32(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 rn_pack8(const float (&f)[8])
{
    return make_uint4(rn_pack2(f[0], f[1]), rn_pack2(f[2], f[3]), rn_pack2(f[4], f[5]), rn_pack2(f[6], f[7]));
}

template <bool FP32>
__device__ __forceinline__ void rn_load_stream(const void *p, size_t off, float (&f)[8])
{
    if constexpr (FP32) {
        const float4 a = *reinterpret_cast<const float4 *>((const float *)p + off);
        const float4 b = *reinterpret_cast<const float4 *>((const float *)p + off + 4);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        rn_unpack8(*reinterpret_cast<const uint4 *>((const uint16_t *)p + off), f);
    }
}

// Sum over the T threads of a row; every thread gets it.  The order is fixed.
template <int T>
__device__ __forceinline__ float rn_row_sum(float v, float *red)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    if constexpr (T > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < T / 64; ++w) v += red[w];
        __syncthreads();
    }
    return v;
}

template <int C>
__device__ __forceinline__ void rn_clear(float (&v)[C][8], const bool (&in)[C])
{
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = in[c] ? v[c][i] : 0.0f;
}

template <int C>
__device__ __forceinline__ void rn_raw(uint4 (&u)[C], const uint16_t *p, const int (&k)[C])
{
#pragma unroll
    for (int c = 0; c < C; ++c) u[c] = *reinterpret_cast<const uint4 *>(p + k[c]);
}

template <int C>
__device__ __forceinline__ void rn_times(float (&v)[C][8], const uint16_t *p, const int (&k)[C])
{
    uint4 u[C];
    rn_raw<C>(u, p, k);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float f[8];
        rn_unpack8(u[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= f[i];
    }
}

template <int C>
__device__ __forceinline__ void rn_plus(float (&v)[C][8], const uint16_t *p, const int (&k)[C])
{
    uint4 u[C];
    rn_raw<C>(u, p, k);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float f[8];
        rn_unpack8(u[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += f[i];
    }
}

// v <- v / sqrt(mean(v^2) + eps), centred first for LayerNorm.  Elements past
// D are zero on entry and stay out of the sums.
template <int T, int C>
__device__ __forceinline__ void rn_normalize(float (&v)[C][8], int kind, const bool (&in)[C], float inv_d, float eps,
                                             float *red)
{
    if (kind == SVDQ_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[c][i];
        const float mean = rn_row_sum<T>(s, red) * inv_d;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = in[c] ? v[c][i] - mean : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) q = __builtin_fmaf(v[c][i], v[c][i], q);
    const float rs = 1.0f / __builtin_sqrtf(rn_row_sum<T>(q, red) * inv_d + eps);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= rs;
}

// T threads per row (64: four rows per block of 256), C chunks of 8 channels
// per thread: chunk c of thread t is channels 8 (t + c T) .. + 7.
template <int T, int C, bool FP32>
__global__ __launch_bounds__(T < 256 ? 256 : T) void residual_norm_kernel(ResidualNormArgs a)
{
    __shared__ float red[T < 256 ? 1 : T / 64];
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    const int t = threadIdx.x % T;
    const int m = (int)(blockIdx.y * a.grid_x + blockIdx.x) * ROWS + threadIdx.x / T;
    if (m >= a.M) return;                           // whole waves (T = 64) or none (one row per block)
    const int D = a.D;
    const float inv_d = 1.0f / (float)D;
    const size_t row = (size_t)m * D;
    int b = a.mod_index ? a.mod_index[m] : m / a.rows_per_mod;
    const bool mod = (uint32_t)b < (uint32_t)a.mod_rows;
    const size_t mrow = mod ? (size_t)b * a.mod_stride : 0;

    // loads carry no condition (a condition makes the compiler wait for one
    // load before the next): chunks past D repeat the last one, count as zero
    // and are not stored
    int k[C];
    bool in[C];
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = 8 * (t + c * T) < D, k[c] = min(8 * (t + c * T), D - 8);
    float v[C][8];
    if (a.y) {
        float r[C][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            rn_unpack8(*reinterpret_cast<const uint4 *>(a.y + row + k[c]), v[c]);
            rn_load_stream<FP32>(a.r, row + k[c], r[c]);
        }
        rn_clear<C>(v, in);
        if (a.post != SVDQ_NORM_NONE) rn_normalize<T, C>(v, a.post, in, inv_d, a.eps, red);
        if (a.post_w) rn_times<C>(v, a.post_w, k);
        if (a.gate && mod) rn_times<C>(v, a.gate + mrow, k);
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = __builtin_fmaf(a.alpha, v[c][i], r[c][i]);
            if (!in[c]) continue;
            if constexpr (FP32) {
                float *o = (float *)a.r_out + row + k[c];
                *reinterpret_cast<float4 *>(o) = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
                *reinterpret_cast<float4 *>(o + 4) = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
            } else {
                *reinterpret_cast<uint4 *>((uint16_t *)a.r_out + row + k[c]) = rn_pack8(v[c]);
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) rn_load_stream<FP32>(a.r, row + k[c], v[c]);
    }
    rn_clear<C>(v, in);
    if (!a.x) return;
    if (a.pre != SVDQ_NORM_NONE) rn_normalize<T, C>(v, a.pre, in, inv_d, a.eps, red);
    if (a.pre_w) rn_times<C>(v, a.pre_w, k);
    if (a.pre_b) rn_plus<C>(v, a.pre_b, k);
    if (a.scale && mod) {
        uint4 u[C];
        rn_raw<C>(u, a.scale + mrow, k);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float f[8];
            rn_unpack8(u[c], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = __builtin_fmaf(v[c][i], f[i], v[c][i]);
        }
    }
    if (a.shift && mod) rn_plus<C>(v, a.shift + mrow, k);
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (in[c]) *reinterpret_cast<uint4 *>(a.x + row + k[c]) = rn_pack8(v[c]);
}

template <int T, int C>
hipError_t rn_launch(ResidualNormArgs a, bool fp32, hipStream_t stream)
{
    const int rows = T < 256 ? 256 / T : 1;
    const LaunchGrid g = launch_grid(((int64_t)a.M + rows - 1) / rows);
    const dim3 grid(g.x, g.y), block(T < 256 ? 256 : T);
    a.grid_x = (int)g.x;
    if (fp32) residual_norm_kernel<T, C, true><<<grid, block, 0, stream>>>(a);
    else residual_norm_kernel<T, C, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(const ResidualNormArgs &a, bool fp32, hipStream_t stream)
{
    const int D = a.D;
    if (D <= 512) return rn_launch<64, 1>(a, fp32, stream);
    if (D <= 1024) return rn_launch<64, 2>(a, fp32, stream);
    if (D <= 2048) return rn_launch<256, 1>(a, fp32, stream);
    if (D <= 4096) return rn_launch<256, 2>(a, fp32, stream);
    if (D <= 8192) return rn_launch<256, 4>(a, fp32, stream);
    return rn_launch<256, 8>(a, fp32, stream);
}

}  // namespace svdq
