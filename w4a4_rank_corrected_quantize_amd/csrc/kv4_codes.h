// kv4_codes.h -- quantizing a tile of tokens' keys and values into the pages of
// the 4-bit cache, shared by the kernels that write it (kv4_cache.hip,
// rope.hip).  Those files are compiled with -ffp-contract=off: the codes are
// bit-exact by contract.
#pragma once

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

// LDS of a tile: one head of 2048 / D consecutive tokens.
template <int D>
struct KcTile {
    static constexpr int TB = 2048 / D;         // tokens
    __attribute__((aligned(16))) uint8_t vt[D / 2][TB + 4];
    int sl[TB];                                 // slots, -1 for none
};

// Quantizes a tile and writes it: thread q = tid % (D / 8) of token tid / (D /
// 8) has channels 8 q .. of the token's key (fk) and value (fv).  The block's
// threads all call it; m.sl is written before (a barrier between).
template <bool INT4, int D>
__device__ __forceinline__ void kc_store_tile(const Kv4View &c, int head, KcTile<D> &m, const float (&fk)[8],
                                              const float (&fv)[8], int tid)
{
    constexpr int TPT = D / 8;                  // threads per token
    constexpr int TB = KcTile<D>::TB;
    const int tk = tid / TPT, q = tid % TPT;
    const int P = 1 << c.page_shift;
    auto &vt = m.vt;
    auto &sl = m.sl;
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

}  // namespace
}  // namespace svdq
