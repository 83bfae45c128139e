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

// The top bytes of four floats.
__device__ __forceinline__ uint32_t kc_top_bytes(const float *f)
{
    return __builtin_amdgcn_perm(f32_bits(f[1]), f32_bits(f[0]), 0x0c0c0703u) |
           __builtin_amdgcn_perm(f32_bits(f[3]), f32_bits(f[2]), 0x07030c0cu);
}

template <int CTRL>
__device__ __forceinline__ float kc_dpp(float x)
{
    return bits_f32(__builtin_amdgcn_update_dpp(0, f32_bits(x), CTRL, 0xF, 0xF, true));
}

// The group's largest magnitude; the group is 8 (INT4) or 4 (MXFP4) neighbouring lanes of 8
// channels each.
template <bool INT4>
__device__ __forceinline__ float kc_absmax(const float (&f)[8])
{
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, __builtin_fabsf(f[i]));
    a = fmaxf(a, kc_dpp<0xB1>(a));                      // lane ^ 1
    a = fmaxf(a, kc_dpp<0x4E>(a));                      // lane ^ 2
    if (INT4) a = fmaxf(a, kc_dpp<0x141>(a));           // the other four of eight (mirrored)
    return a;
}

// Stored scales are finite, so that a place that a row does not see (weight 0)
// cannot reach it: a group that holds an infinity is stored as zeros (INT4) or
// with 6 * 2^125 for it (MXFP4; 2^125 is the largest scale that finite bf16
// values give).
__device__ __forceinline__ float kc_finite(float scale) { return scale < INFINITY ? scale : 0.0f; }
__device__ __forceinline__ uint32_t kc_finite(uint32_t e8m0) { return min(e8m0, 252u); }

// The low bytes of four words.
__device__ __forceinline__ uint32_t kc_low_bytes(const uint32_t *w)
{
    return __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400u) | __builtin_amdgcn_perm(w[3], w[2], 0x04000c0cu);
}

// Codes of 8 channels, byte i channel i (low nibble) and i + 4 (high).  |q| =
// rint(|v| / scale): added to 1.5 2^23 the product with the reciprocal leaves
// q in the sum's low bits.  The remainder |v| - q scale is exact in one fma, and
// q is right wherever it lies strictly within half the scale; a group with one
// that does not (the reciprocal's error, and ties: bf16 values meet these often,
// one group in seven has a scale that is exact in few bits) moves it by one.
__device__ __forceinline__ uint32_t kc_int4_codes(const float (&f)[8], float scale)
{
    constexpr float kMagic = 12582912.0f;
    uint32_t q[8];
    if (scale < 7.88860905e-31f) {                      // 2^-100: the exact path's lift
        const Int4Group g = int4_group_prepare(scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = int4_mag(__builtin_fabsf(f[i]), g);
    } else {
        const float inv = __builtin_amdgcn_rcpf(scale), half = 0.5f * scale;
        float e[8], far = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float m = __builtin_fmaf(__builtin_fabsf(f[i]), inv, kMagic);
            e[i] = __builtin_fmaf(kMagic - m, scale, __builtin_fabsf(f[i]));
            q[i] = f32_bits(m);
            far = fmaxf(far, __builtin_fabsf(e[i]));
        }
        if (far >= half) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float h = bits_f32(f32_bits(half) - (q[i] & 1u));     // an odd q loses a tie
                q[i] += (uint32_t)(e[i] > h) - (uint32_t)(e[i] < -h);
            }
        }
    }
    return kc_low_bytes(q) | (kc_low_bytes(q + 4) << 4) | ((kc_top_bytes(f) >> 4) & 0x08080808u) |
           (kc_top_bytes(f + 4) & 0x80808080u);
}

// The conversion instruction rounds v / 2^X (exact) to the E2M1 grid, ties to
// the even index, saturates at 6 and keeps the sign of zero.  SPLIT: byte i
// holds channels i and i + 4, else 2 i and 2 i + 1.
template <bool SPLIT>
__device__ __forceinline__ uint32_t kc_e2m1_codes(const float (&f)[8], float inv)
{
    constexpr int A = SPLIT ? 1 : 2, B = SPLIT ? 4 : 1;
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0] * inv, f[B] * inv, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[A] * inv, f[A + B] * inv, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2 * A] * inv, f[2 * A + B] * inv, 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[3 * A] * inv, f[3 * A + B] * inv, 1.0f, 3);
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
    __shared__ __attribute__((aligned(16))) uint8_t vt[D / 2][TB + 4];
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
    const float ka = kc_absmax<INT4>(fk), va = kc_absmax<INT4>(fv);
    float ks = 0.0f, vs = 0.0f;
    uint32_t ke = 0, ve = 0, kw, vw;
    if constexpr (INT4) {
        ks = kc_finite(int4_group_scale(ka)), vs = kc_finite(int4_group_scale(va));
        kw = kc_int4_codes(fk, ks), vw = kc_int4_codes(fv, vs);
    } else {
        ke = kc_finite(mx_block_e8m0(ka)), ve = kc_finite(mx_block_e8m0(va));
        kw = kc_e2m1_codes<false>(fk, mx_inv_scale(ke)), vw = kc_e2m1_codes<true>(fv, mx_inv_scale(ve));
    }
    // channels 8 q .. of a 32-block: parts 0, 1 are low nibbles, 2, 3 high
    const uint32_t other = __shfl_xor(vw, 2);
    if ((q & 2) == 0) {
        const uint32_t lo = (vw & 0x0F0F0F0Fu) | ((other << 4) & 0xF0F0F0F0u);
        const uint32_t hi = ((vw >> 4) & 0x0F0F0F0Fu) | (other & 0xF0F0F0F0u);
        uint8_t (*r)[TB + 4] = vt + 16 * (q >> 2) + 8 * (q & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i][tk] = (uint8_t)(lo >> (8 * i)), r[i + 4][tk] = (uint8_t)(hi >> (8 * i));
    }
    size_t page;
    int place;
    if (kc_slot(c, sl[tk], page, place)) {
        const size_t run = ((page * c.heads + head) * P + place) >> 4;
        *reinterpret_cast<uint32_t *>(c.k_codes + run * (8 * D) + kv4_k_offset<INT4>(place & 15, 8 * q, D)) = kw;
        constexpr int G = INT4 ? 64 : 32;
        if ((8 * q) % G == 0) {
            const size_t o = run * (16 * D / G) + 16 * (8 * q / G) + (place & 15);
            if constexpr (INT4) ((float *)c.k_scales)[o] = ks, ((float *)c.v_scales)[o] = vs;
            else ((uint8_t *)c.k_scales)[o] = (uint8_t)ke, ((uint8_t *)c.v_scales)[o] = (uint8_t)ve;
        }
    }
    __syncthreads();
    // four tokens at a time: a dword where their slots are consecutive and
    // aligned, else bytes
    const int g4 = 4 * (tid % (TB / 4));
    const int s0 = sl[g4];
    const bool quad = (s0 & 3) == 0 && sl[g4 + 1] == s0 + 1 && sl[g4 + 2] == s0 + 2 && sl[g4 + 3] == s0 + 3;
    if (quad) {
        if (kc_slot(c, s0, page, place)) {
            uint8_t *run = c.v_codes + (((page * c.heads + head) * P + place) >> 4) * (8 * D);
            for (int r = tid / (TB / 4); r < D / 2; r += 4 * TPT)
                *reinterpret_cast<uint32_t *>(run + kv4_v_offset(place & 15, r >> 4, r & 15, D)) =
                    *reinterpret_cast<const uint32_t *>(&vt[r][g4]);
        }
    } else {
        for (int i = 0; i < 4; ++i) {
            if (!kc_slot(c, sl[g4 + i], page, place)) continue;
            uint8_t *run = c.v_codes + (((page * c.heads + head) * P + place) >> 4) * (8 * D);
            for (int r = tid / (TB / 4); r < D / 2; r += 4 * TPT)
                run[kv4_v_offset(place & 15, r >> 4, r & 15, D)] = vt[r][g4 + i];
        }
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
