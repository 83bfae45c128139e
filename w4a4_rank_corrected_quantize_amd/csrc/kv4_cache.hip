// kv4_cache.hip -- writing tokens into the 4-bit key / value cache and
// reading them back.
//
// Codes and scales are those of the library's group quantizers (svdq_quant.h)
// along the head's channels, bit for bit.  Bound by HBM: append reads 4 bytes
// (K and V in bf16) and writes about 1.1 bytes per channel, read the reverse
// with fp32 values.  4608 tokens, 32 heads of 64, INT4: 13 us for 48 MB and 16
// us for 86 MB (3.7 and 5.4 TB/s), MXFP4 11 and 17 us; 1024 tokens, 24 heads of
// 128, MXFP4: 4.5 and 8.6 us.  Append is held by the quantizer's arithmetic next to the loads
// (about 120 vector instructions per 8 channels of K and as many of V).
//
// A block takes one head of 2048 / D consecutive tokens, 8 channels per
// thread.  K codes are written as they come out, one dword per thread; V codes
// are turned in LDS so that four lanes write the bytes of four tokens, which
// form a dword where the slots are consecutive.
#include "kv4_codes.h"

namespace svdq {
namespace {

template <bool INT4, int D>
__global__ __launch_bounds__(KC_THREADS) void kv4_append_kernel(Kv4View c, const uint16_t *__restrict__ K,
                                                                const uint16_t *__restrict__ V, int64_t ldk,
                                                                int64_t ldv, const int32_t *__restrict__ slots, int T)
{
    constexpr int TPT = D / 8;                  // threads per token
    constexpr int TB = KcTile<D>::TB;           // tokens per block
    __shared__ KcTile<D> m;
    const int tid = threadIdx.x, tk = tid / TPT, q = tid % TPT;
    const int head = blockIdx.x % c.heads, t0 = (int)(blockIdx.x / c.heads) * TB;
    if (tid < TB) m.sl[tid] = t0 + tid < T ? slots[t0 + tid] : -1;
    float fk[8], fv[8];
    const int t = min(t0 + tk, T - 1);
    kc_unpack8(*reinterpret_cast<const uint4 *>(K + t * ldk + head * D + 8 * q), fk);
    kc_unpack8(*reinterpret_cast<const uint4 *>(V + t * ldv + head * D + 8 * q), fv);
    __syncthreads();
    kc_store_tile<INT4, D>(c, head, m, fk, fv, tid);
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

// A slot outside the cache reads as zeros.  A thread has four channels of two
// tokens, so that a wave's stores are whole lines.
template <bool INT4, int D>
__global__ __launch_bounds__(KC_THREADS) void kv4_read_kernel(Kv4View c, const int32_t *__restrict__ slots, int T,
                                                              float *__restrict__ K, float *__restrict__ V)
{
    constexpr int TPT = D / 8;
    constexpr int TB = KC_THREADS / TPT;
    constexpr int G = INT4 ? 64 : 32;
    __shared__ __attribute__((aligned(16))) uint8_t vt[D / 2][TB + 4];
    __shared__ int sl[TB];
    const int tid = threadIdx.x;
    const int head = blockIdx.x % c.heads, t0 = (int)(blockIdx.x / c.heads) * TB;
    const int P = 1 << c.page_shift;
    if (tid < TB) sl[tid] = t0 + tid < T ? slots[t0 + tid] : -1;
    // K's codes and the scales, on their way while V's codes go through LDS
    const int ch = 4 * (tid % (D / 4));
    size_t page;
    int place;
    bool mine[2];
    uint32_t w[2];
    float ks[2], vs[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = t0 + tid / (D / 4) + h * (TB / 2);
        mine[h] = kc_slot(c, t < T ? slots[t] : -1, page, place);
        const size_t run = mine[h] ? ((page * c.heads + head) * P + place) >> 4 : 0;        // run 0 exists
        const int tok = mine[h] ? place & 15 : 0;
        w[h] = *reinterpret_cast<const uint32_t *>(c.k_codes + run * (8 * D) + kv4_k_offset<INT4>(tok, ch & ~7, D));
        const size_t so = run * (16 * D / G) + 16 * (ch / G) + tok;
        if constexpr (INT4) ks[h] = ((const float *)c.k_scales)[so], vs[h] = ((const float *)c.v_scales)[so];
        else ks[h] = kv4_e8m0(((const uint8_t *)c.k_scales)[so]), vs[h] = kv4_e8m0(((const uint8_t *)c.v_scales)[so]);
    }
    __syncthreads();
    const int g4 = 4 * (tid % (TB / 4));
    const int s0 = sl[g4];
    const bool quad = (s0 & 3) == 0 && sl[g4 + 1] == s0 + 1 && sl[g4 + 2] == s0 + 2 && sl[g4 + 3] == s0 + 3;
    if (quad) {
        if (kc_slot(c, s0, page, place)) {
            const uint8_t *vr = c.v_codes + (((page * c.heads + head) * P + place) >> 4) * (8 * D);
#pragma unroll
            for (int i = 0; i < D / 2 / (4 * TPT); ++i) {
                const int r = tid / (TB / 4) + 4 * TPT * i;
                *reinterpret_cast<uint32_t *>(&vt[r][g4]) =
                    *reinterpret_cast<const uint32_t *>(vr + kv4_v_offset(place & 15, r >> 4, r & 15, D));
            }
        }
    } else {
        for (int i = 0; i < 4; ++i) {
            if (!kc_slot(c, sl[g4 + i], page, place)) continue;
            const uint8_t *vr = c.v_codes + (((page * c.heads + head) * P + place) >> 4) * (8 * D);
            for (int r = tid / (TB / 4); r < D / 2; r += 4 * TPT)
                vt[r][g4 + i] = vr[kv4_v_offset(place & 15, r >> 4, r & 15, D)];
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int tk = tid / (D / 4) + h * (TB / 2);
        if (t0 + tk >= T) continue;
        float fk[4] = {}, fv[4] = {};
        if (mine[h]) {
            const int row = 16 * (ch >> 5) + (ch & 15), vsh = (ch >> 4) & 1 ? 4 : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ksh = INT4 ? 8 * i + (ch & 4) : 4 * (i + (ch & 4));
                fk[i] = kc_value((w[h] >> ksh) & 15u, ks[h], INT4);
                fv[i] = kc_value((uint32_t)(vt[row + i][tk] >> vsh) & 15u, vs[h], INT4);
            }
        }
        const size_t o = ((size_t)(t0 + tk) * c.heads + head) * D + ch;
        *reinterpret_cast<float4 *>(K + o) = make_float4(fk[0], fk[1], fk[2], fk[3]);
        *reinterpret_cast<float4 *>(V + o) = make_float4(fv[0], fv[1], fv[2], fv[3]);
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
