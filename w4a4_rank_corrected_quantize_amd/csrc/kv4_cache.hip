// kv4_cache.hip -- writing tokens into the 4-bit key / value cache and
// reading them back.
//
// Codes and scales are those of the library's group quantizers (svdq_quant.h)
// along the head's channels, bit for bit.  Bound by HBM: append reads 4 bytes
// (K and V in bf16) and writes about 1.1 bytes per channel.
//
// A block takes one head of 2048 / D consecutive tokens, 8 channels per
// thread.  K codes are written as they come out, one dword per thread; V codes
// are turned in LDS so that four lanes write the bytes of four tokens, which
// form a dword where the slots are consecutive.
#include "kv4.h"

namespace svdq {
namespace {

constexpr int KC_THREADS = 256;

__device__ __forceinline__ void kc_unpack8(const uint4 &u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bits_f32(w[i] << 16);
        f[2 * i + 1] = bits_f32(w[i] & 0xFFFF0000u);
    }
}

// Codes of 8 channels (element i in nibble i of `natural`) and the group's
// scale; the group is 8 (INT4) or 4 (MXFP4) neighbouring lanes.
template <bool INT4>
__device__ __forceinline__ uint32_t kc_quantize8(const float (&f)[8], float &scale, uint32_t &e8m0)
{
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, __builtin_fabsf(f[i]));
#pragma unroll
    for (int d = 1; d < (INT4 ? 8 : 4); d <<= 1) a = fmaxf(a, __shfl_xor(a, d));
    uint32_t w = 0;
    if constexpr (INT4) {
        scale = int4_group_scale(a);
        const Int4Group g = int4_group_prepare(scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= int4_nibble(f[i], g) << (4 * i);
    } else {
        e8m0 = mx_block_e8m0(a);
        const float inv = mx_inv_scale(e8m0);
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= e2m1_code(f[i], inv) << (4 * i);
    }
    return w;
}

// nibbles 0 .. 7 -> byte i holds element i (low) and i + 4 (high)
__device__ __forceinline__ uint32_t kc_interleave(uint32_t w)
{
    uint32_t lo = w & 0xFFFFu, hi = w >> 16;
    lo = (lo | (lo << 8)) & 0x00FF00FFu, lo = (lo | (lo << 4)) & 0x0F0F0F0Fu;
    hi = (hi | (hi << 8)) & 0x00FF00FFu, hi = (hi | (hi << 4)) & 0x0F0F0F0Fu;
    return lo | (hi << 4);
}

__device__ __forceinline__ uint32_t kc_deinterleave(uint32_t w)
{
    uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
    lo = (lo | (lo >> 4)) & 0x00FF00FFu, lo = (lo | (lo >> 8)) & 0xFFFFu;
    hi = (hi | (hi >> 4)) & 0x00FF00FFu, hi = (hi | (hi >> 8)) & 0xFFFFu;
    return lo | (hi << 16);
}

// A slot's page and place, false outside the cache.
__device__ __forceinline__ bool kc_slot(const Kv4View &c, int slot, size_t &page, int &place)
{
    if (slot < 0 || slot >= c.pages << c.page_shift) return false;
    page = (size_t)(slot >> c.page_shift);
    place = slot & ((1 << c.page_shift) - 1);
    return true;
}

template <bool INT4, int D>
__global__ __launch_bounds__(KC_THREADS) void kv4_append_kernel(Kv4View c, const uint16_t *__restrict__ K,
                                                                const uint16_t *__restrict__ V, int64_t ldk,
                                                                int64_t ldv, const int32_t *__restrict__ slots, int T)
{
    constexpr int TPT = D / 8;                  // threads per token
    constexpr int TB = KC_THREADS / TPT;        // tokens per block
    __shared__ uint8_t vt[D / 2][TB + 4];
    __shared__ int sl[TB];
    const int tid = threadIdx.x, tk = tid / TPT, q = tid % TPT;
    const int head = blockIdx.x % c.heads, t0 = (int)(blockIdx.x / c.heads) * TB;
    const int P = 1 << c.page_shift;
    if (tid < TB) sl[tid] = t0 + tid < T ? slots[t0 + tid] : -1;
    float fk[8], fv[8];
    const int t = min(t0 + tk, T - 1);
    kc_unpack8(*reinterpret_cast<const uint4 *>(K + t * ldk + head * D + 8 * q), fk);
    kc_unpack8(*reinterpret_cast<const uint4 *>(V + t * ldv + head * D + 8 * q), fv);
    __syncthreads();
    float ks = 0.0f, vs = 0.0f;
    uint32_t ke = 0, ve = 0;
    const uint32_t kw = kc_quantize8<INT4>(fk, ks, ke), vw = kc_quantize8<INT4>(fv, vs, ve);
    // channels 8 q .. of a 32-block: parts 0, 1 are low nibbles, 2, 3 high
    const uint32_t other = __shfl_xor(vw, 2);
    if ((q & 2) == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            vt[16 * (q >> 2) + 8 * (q & 1) + i][tk] =
                (uint8_t)(((vw >> (4 * i)) & 15u) | (((other >> (4 * i)) & 15u) << 4));
    }
    size_t page;
    int place;
    if (kc_slot(c, sl[tk], page, place)) {
        const size_t run = ((page * c.heads + head) * P + place) >> 4;
        const uint32_t w = INT4 ? kc_interleave(kw) : kw;
        *reinterpret_cast<uint32_t *>(c.k_codes + run * (8 * D) + kv4_k_offset<INT4>(place & 15, 8 * q, D)) = w;
        constexpr int G = INT4 ? 64 : 32;
        if ((8 * q) % G == 0) {
            const size_t o = run * (16 * D / G) + 16 * (8 * q / G) + (place & 15);
            if constexpr (INT4) ((float *)c.k_scales)[o] = ks, ((float *)c.v_scales)[o] = vs;
            else ((uint8_t *)c.k_scales)[o] = (uint8_t)ke, ((uint8_t *)c.v_scales)[o] = (uint8_t)ve;
        }
    }
    __syncthreads();
    const int vtk = tid % TB;
    if (kc_slot(c, sl[vtk], page, place)) {
        uint8_t *run = c.v_codes + (((page * c.heads + head) * P + place) >> 4) * (8 * D);
        for (int r = tid / TB; r < D / 2; r += TPT) run[kv4_v_offset(place & 15, r >> 4, r & 15, D)] = vt[r][vtk];
    }
}

__device__ __forceinline__ float kc_value(uint32_t code, float scale, bool int4)
{
    const uint32_t m = code & 7u;
    float v;
    if (int4) {
        v = (float)m;
    } else {
        // E2M1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
        v = m < 2 ? 0.5f * (float)m : bits_f32(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    }
    v *= scale;
    return code & 8u ? -v : v;
}

// A slot outside the cache reads as zeros.
template <bool INT4, int D>
__global__ __launch_bounds__(KC_THREADS) void kv4_read_kernel(Kv4View c, const int32_t *__restrict__ slots, int T,
                                                              float *__restrict__ K, float *__restrict__ V)
{
    constexpr int TPT = D / 8;
    constexpr int TB = KC_THREADS / TPT;
    constexpr int G = INT4 ? 64 : 32;
    __shared__ uint8_t vt[D / 2][TB + 4];
    __shared__ int sl[TB];
    const int tid = threadIdx.x, tk = tid / TPT, q = tid % TPT;
    const int head = blockIdx.x % c.heads, t0 = (int)(blockIdx.x / c.heads) * TB;
    const int P = 1 << c.page_shift;
    if (tid < TB) sl[tid] = t0 + tid < T ? slots[t0 + tid] : -1;
    __syncthreads();
    size_t page;
    int place;
    const int vtk = tid % TB;
    if (kc_slot(c, sl[vtk], page, place)) {
        const uint8_t *run = c.v_codes + (((page * c.heads + head) * P + place) >> 4) * (8 * D);
        for (int r = tid / TB; r < D / 2; r += TPT) vt[r][vtk] = run[kv4_v_offset(place & 15, r >> 4, r & 15, D)];
    }
    __syncthreads();
    if (t0 + tk >= T) return;
    float fk[8] = {}, fv[8] = {};
    if (kc_slot(c, sl[tk], page, place)) {
        const size_t run = ((page * c.heads + head) * P + place) >> 4;
        uint32_t w = *reinterpret_cast<const uint32_t *>(c.k_codes + run * (8 * D) + kv4_k_offset<INT4>(place & 15, 8 * q, D));
        if (INT4) w = kc_deinterleave(w);
        const size_t o = run * (16 * D / G) + 16 * (8 * q / G) + (place & 15);
        float ks, vs;
        if constexpr (INT4) ks = ((const float *)c.k_scales)[o], vs = ((const float *)c.v_scales)[o];
        else ks = kv4_e8m0(((const uint8_t *)c.k_scales)[o]), vs = kv4_e8m0(((const uint8_t *)c.v_scales)[o]);
        const int sh = q & 2 ? 4 : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            fk[i] = kc_value((w >> (4 * i)) & 15u, ks, INT4);
            fv[i] = kc_value((uint32_t)(vt[16 * (q >> 2) + 8 * (q & 1) + i][tk] >> sh) & 15u, vs, INT4);
        }
    }
    const size_t o = ((size_t)(t0 + tk) * c.heads + head) * D + 8 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<float4 *>(K + o + 4 * h) = make_float4(fk[4 * h], fk[4 * h + 1], fk[4 * h + 2], fk[4 * h + 3]);
        *reinterpret_cast<float4 *>(V + o + 4 * h) = make_float4(fv[4 * h], fv[4 * h + 1], fv[4 * h + 2], fv[4 * h + 3]);
    }
}

}  // namespace

hipError_t launch_kv4_append(const Kv4View &c, const uint16_t *K, const uint16_t *V, int64_t ldk, int64_t ldv,
                             const int32_t *slots, int T, hipStream_t stream)
{
    const int tb = 2048 / c.dim;
    const dim3 grid((uint32_t)((T + tb - 1) / tb) * c.heads);
    if (c.int4 && c.dim == 64) kv4_append_kernel<true, 64><<<grid, KC_THREADS, 0, stream>>>(c, K, V, ldk, ldv, slots, T);
    else if (c.int4) kv4_append_kernel<true, 128><<<grid, KC_THREADS, 0, stream>>>(c, K, V, ldk, ldv, slots, T);
    else if (c.dim == 64) kv4_append_kernel<false, 64><<<grid, KC_THREADS, 0, stream>>>(c, K, V, ldk, ldv, slots, T);
    else kv4_append_kernel<false, 128><<<grid, KC_THREADS, 0, stream>>>(c, K, V, ldk, ldv, slots, T);
    return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4View &c, const int32_t *slots, int T, float *K, float *V, hipStream_t stream)
{
    const int tb = 2048 / c.dim;
    const dim3 grid((uint32_t)((T + tb - 1) / tb) * c.heads);
    if (c.int4 && c.dim == 64) kv4_read_kernel<true, 64><<<grid, KC_THREADS, 0, stream>>>(c, slots, T, K, V);
    else if (c.int4) kv4_read_kernel<true, 128><<<grid, KC_THREADS, 0, stream>>>(c, slots, T, K, V);
    else if (c.dim == 64) kv4_read_kernel<false, 64><<<grid, KC_THREADS, 0, stream>>>(c, slots, T, K, V);
    else kv4_read_kernel<false, 128><<<grid, KC_THREADS, 0, stream>>>(c, slots, T, K, V);
    return hipGetLastError();
}

}  // namespace svdq
