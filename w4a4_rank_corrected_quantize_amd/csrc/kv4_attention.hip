// kv4_attention.hip -- attention of new rows over the 4-bit cache:
//
//   o_i = sum_j p_ij vhat_j / sum_j p_ij,   p_ij = exp(scale q_i . khat_j - max)
//
// over the keys j < kv_len that row i may see (causal: up to its own place;
// window: the last `window` of those), khat and vhat the values the cache
// holds.  Codes become bf16 exactly (q of INT4, q 2^e of MXFP4) and feed the
// bf16 matrix cores; sums, maxima and the softmax are fp32.
//
// The products are formed transposed, S^T = K Q^T and O^T = V^T P^T, with
// v_mfma_f32_16x16x32_bf16: a lane's column is a query row, so maximum, sum
// and rescaling are per lane.  In a step of 64 keys, row r of K tile t is key
// 16 (r / 4) + 4 t + r % 4: lane part b then holds the scores of its keys
// 16 b .. 16 b + 15, which are the 16 tokens that it reads of V, so the
// probabilities go from one product to the next in registers.  The page
// layout (kv4.h) gives a lane its part of a K row and its V column as 16-byte
// loads in operand order; nothing passes through LDS.
//
// INT4 scales (fp32) belong to a key and a 64-channel group: a lane holds the
// scale of key 16 b + lane % 16 and multiplies with a row broadcast (DPP).
// K's multiply the group's score sums, V's the probabilities before they are
// rounded to bf16.  MXFP4 scales enter the fp4 -> bf16 conversion itself.
//
// Rounding choices: p (INT4: p times V's scale) is rounded to bf16 for the
// second product (at most 2^-8 relative, as the output's own type rounds);
// the sum of p is taken of the unrounded values.
//
// Rows are packed: the G = heads_q / heads query heads that share a key head
// and the sequence's new tokens form one list, row = token G + head, so
// single tokens of grouped heads fill the 16 columns of a product.  A block
// of four waves takes 16 CT rows per wave; if the sequence has no more than
// 16 CT rows its waves share them and take every fourth step of keys instead,
// and add up at the end.  Sequences are further split over blocks where the
// grid would not fill the chip; the splits' sums then go to the workspace and
// a second kernel adds them in split order.
#include "kv4.h"

namespace svdq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ uint32_t ka_pack2(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Value of lane J of the lane's row of 16.
template <int J>
__device__ __forceinline__ float ka_row_bcast(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + J, 0xF, 0xF, true));
}

__device__ __forceinline__ float ka_max_parts(float x)     // over the four lane parts
{
    auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    x = fmaxf(bits_f32(a[0]), bits_f32(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return fmaxf(bits_f32(b[0]), bits_f32(b[1]));
}

__device__ __forceinline__ float ka_sum_parts(float x)
{
    auto a = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    x = bits_f32(a[0]) + bits_f32(a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return bits_f32(b[0]) + bits_f32(b[1]);
}

// Codes to bf16.  INT4: sign-magnitude nibbles become the fp8 (E4M3) bytes of
// q 2^-9, converted with the factor 2^9.
__device__ __forceinline__ uint32_t ka_e4m3_low(uint32_t w) { return (w & 0x07070707u) | ((w << 4) & 0x80808080u); }
__device__ __forceinline__ uint32_t ka_e4m3_high(uint32_t w) { return ((w >> 4) & 0x07070707u) | (w & 0x80808080u); }

template <bool HIGH>
__device__ __forceinline__ uint32_t ka_cvt_fp8(uint32_t w)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 512.0f, HIGH));
}

template <int BYTE>
__device__ __forceinline__ uint32_t ka_cvt_fp4(uint32_t w, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, BYTE));
}

struct KvArgs {
    Kv4View c;
    const uint16_t *Q;
    const int32_t *table, *q_start, *kv_len;
    uint16_t *O;
    float *lse, *work;
    int64_t ldq;
    int T, B, heads_q, group, table_width, q_tiles, splits, causal, window;
    float scale;
};

// One step's codes and scales in flight.
template <int D, bool INT4>
struct KvStep {
    static constexpr int KS = D / 32;             // 32-channel product steps = dwords of a lane's K part
    static constexpr int NB = D / 32;             // 32-channel blocks of V
    static constexpr int NG = INT4 ? D / 64 : D / 32;
    uint32_t k[4][KS];
    u32x4 v[NB];
    float ks[INT4 ? NG : 4];                      // INT4: of key 16 b + lane % 16; MXFP4: of the K row of tile t
    float vs[NG];                                 // of key 16 b + lane % 16
    bool ok;                                      // the lane part's 16 keys lie in a page of the cache
};

template <int D, bool INT4>
__device__ __forceinline__ void ka_load(KvStep<D, INT4> &st, const KvArgs &a, const int32_t *table, int head, int key0,
                                        int kv_end, int lane)
{
    constexpr int NB = D / 32, NG = KvStep<D, INT4>::NG;
    const int P = 1 << a.c.page_shift, j = lane & 15, b = lane >> 4;
    // page of the 16 keys that hold the lane's K rows, and of its V columns
    const int runk = key0 + 16 * (j >> 2), runv = key0 + 16 * b;
    int pk = runk < kv_end ? table[runk >> a.c.page_shift] : -1;
    int pv = runv < kv_end ? table[runv >> a.c.page_shift] : -1;
    st.ok = (uint32_t)pv < (uint32_t)a.c.pages;
    pk = (uint32_t)pk < (uint32_t)a.c.pages ? pk : 0;       // masked below; page 0 exists
    pv = st.ok ? pv : 0;
    const size_t hk = (size_t)pk * a.c.heads + head, hv = (size_t)pv * a.c.heads + head;
    const int ik = runk & (P - 1), iv = runv & (P - 1);
    const uint8_t *kc = a.c.k_codes + (hk * P + ik + (j & 3)) * (D / 2) + b * (D / 8);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4 *>(kc + 4 * t * (D / 2));
            st.k[t][0] = u.x, st.k[t][1] = u.y, st.k[t][2] = u.z, st.k[t][3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(kc + 4 * t * (D / 2));
            st.k[t][0] = u.x, st.k[t][1] = u.y;
        }
    }
    const uint8_t *vc = a.c.v_codes + (hv * (D / 2) + j) * P + iv;
#pragma unroll
    for (int n = 0; n < NB; ++n) st.v[n] = *reinterpret_cast<const u32x4 *>(vc + (size_t)16 * n * P);
    const bool in = st.ok && runv + j < kv_end;
    if constexpr (INT4) {
        const float *ks = (const float *)a.c.k_scales + hv * NG * P + iv + j;
        const float *vs = (const float *)a.c.v_scales + hv * NG * P + iv + j;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            st.ks[g] = ks[g * P];
            const float s = vs[g * P];
            st.vs[g] = in ? s : 0.0f;             // a place past the end may hold anything: 0, not 0 times that
        }
    } else {
        const int blk = D == 128 ? b : b >> 1;    // the 32-channel block of the lane's K part
        const uint8_t *ks = (const uint8_t *)a.c.k_scales + (hk * NG + blk) * P + ik + (j & 3);
#pragma unroll
        for (int t = 0; t < 4; ++t) st.ks[t] = bits_f32((uint32_t)ks[4 * t] << 23);
        const uint8_t *vs = (const uint8_t *)a.c.v_scales + hv * NG * P + iv + j;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t e = vs[g * P];
            st.vs[g] = in ? bits_f32(e << 23) : 0.0f;
        }
    }
}

// Operand of 8 channels of a K row.
template <bool INT4>
__device__ __forceinline__ bf16x8 ka_k_operand(uint32_t w, float scale)
{
    u32x4 o;
    if constexpr (INT4) {
        const uint32_t lo = ka_e4m3_low(w), hi = ka_e4m3_high(w);
        o = (u32x4){ka_cvt_fp8<false>(lo), ka_cvt_fp8<true>(lo), ka_cvt_fp8<false>(hi), ka_cvt_fp8<true>(hi)};
    } else {
        o = (u32x4){ka_cvt_fp4<0>(w, scale), ka_cvt_fp4<1>(w, scale), ka_cvt_fp4<2>(w, scale), ka_cvt_fp4<3>(w, scale)};
    }
    return __builtin_bit_cast(bf16x8, o);
}

// Operands of 8 keys (two dwords of V codes) for the low- and the high-nibble
// channel.  S: the 8-key half of the lane's 16 keys (for the scales).
template <bool INT4, int S>
__device__ __forceinline__ void ka_v_operands(uint32_t w0, uint32_t w1, float vs, bf16x8 &lo, bf16x8 &hi)
{
    if constexpr (INT4) {
        const uint32_t l0 = ka_e4m3_low(w0), l1 = ka_e4m3_low(w1), h0 = ka_e4m3_high(w0), h1 = ka_e4m3_high(w1);
        lo = __builtin_bit_cast(bf16x8, (u32x4){ka_cvt_fp8<false>(l0), ka_cvt_fp8<true>(l0), ka_cvt_fp8<false>(l1), ka_cvt_fp8<true>(l1)});
        hi = __builtin_bit_cast(bf16x8, (u32x4){ka_cvt_fp8<false>(h0), ka_cvt_fp8<true>(h0), ka_cvt_fp8<false>(h1), ka_cvt_fp8<true>(h1)});
    } else {
        // a byte is one key: its two channels share the key's scale
        uint32_t p[8];
        p[0] = ka_cvt_fp4<0>(w0, ka_row_bcast<8 * S + 0>(vs));
        p[1] = ka_cvt_fp4<1>(w0, ka_row_bcast<8 * S + 1>(vs));
        p[2] = ka_cvt_fp4<2>(w0, ka_row_bcast<8 * S + 2>(vs));
        p[3] = ka_cvt_fp4<3>(w0, ka_row_bcast<8 * S + 3>(vs));
        p[4] = ka_cvt_fp4<0>(w1, ka_row_bcast<8 * S + 4>(vs));
        p[5] = ka_cvt_fp4<1>(w1, ka_row_bcast<8 * S + 5>(vs));
        p[6] = ka_cvt_fp4<2>(w1, ka_row_bcast<8 * S + 6>(vs));
        p[7] = ka_cvt_fp4<3>(w1, ka_row_bcast<8 * S + 7>(vs));
        u32x4 l, h;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u);
            h[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u);
        }
        lo = __builtin_bit_cast(bf16x8, l);
        hi = __builtin_bit_cast(bf16x8, h);
    }
}

// x[4 t + i] *= / += with the scale of key 4 t + i of the lane's part.
template <int J = 0>
__device__ __forceinline__ void ka_scale_keys(float (&o)[16], const float (&x)[16], float s)
{
    if constexpr (J < 16) {
        o[J] = x[J] * ka_row_bcast<J>(s);
        ka_scale_keys<J + 1>(o, x, s);
    }
}

template <int J = 0>
__device__ __forceinline__ void ka_fma_keys(float (&o)[16], const float (&x)[16], float s)
{
    if constexpr (J < 16) {
        o[J] = __builtin_fmaf(x[J], ka_row_bcast<J>(s), o[J]);
        ka_fma_keys<J + 1>(o, x, s);
    }
}

template <int D, bool INT4, int CT>
__global__ __launch_bounds__(256, 2) void kv4_attention_kernel(KvArgs a)
{
    constexpr int KS = D / 32, NB = D / 32, NG = KvStep<D, INT4>::NG;
    constexpr int R = 16 * CT;                        // rows of a wave
    __shared__ float om[R][D + 4];                    // the waves' sums, where they share rows
    __shared__ float mm[4][R], ll[4][R];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j = lane & 15, b = lane >> 4;
    // blocks of one head are consecutive multiples of heads * B apart, so they
    // meet in one XCD's L2 where that is a multiple of 8
    int idx = blockIdx.x;
    const int head = idx % a.c.heads;
    idx /= a.c.heads;
    const int seq = idx % a.B;
    idx /= a.B;
    const int split = idx % a.splits;
    const int qt0 = idx / a.splits;
    const int qs = min(max(a.q_start[seq], 0), a.T);
    const int qn = min(max(a.q_start[seq + 1], qs), a.T) - qs;
    const int kv = min(max(a.kv_len[seq], 0), a.table_width << a.c.page_shift);
    const int32_t *table = a.table + (size_t)seq * a.table_width;
    const int G = a.group;
    const int64_t rows = (int64_t)qn * G;
    const bool shared = rows <= R;                    // one list of rows for the four waves
    const int block_rows = shared ? R : 4 * R;
    const int steps = (kv + 63) >> 6;
    const int per = (steps + a.splits - 1) / a.splits;
    const float c2 = a.scale * kLog2e;

    // the last tiles first: under a causal mask they are the longest
    const int64_t tiles = (rows + block_rows - 1) / block_rows;
    for (int64_t qt = tiles - 1 - qt0; qt >= 0; qt -= a.q_tiles) {
        const int64_t r0 = qt * block_rows + (shared ? 0 : wave * R);
        // Q, limits of every column
        bf16x8 q[CT][KS];
        int hi_key[CT], lo_key[CT];
        int all_hi = kv, any_hi = 0, any_lo = kv, all_lo = 0;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int64_t r = min(r0 + 16 * ct + j, rows - 1);
            const int tok = (int)(r / G), hd = head * G + (int)(r % G);
            const uint16_t *qp = a.Q + (qs + tok) * a.ldq + (int64_t)hd * D;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int ch = INT4 ? 64 * (k >> 1) + 16 * b + 8 * (k & 1) : (D / 4) * b + 8 * k;
                q[ct][k] = *reinterpret_cast<const bf16x8 *>(qp + ch);
            }
            const int place = kv - qn + tok;
            hi_key[ct] = a.causal ? min(place + 1, kv) : kv;
            lo_key[ct] = a.causal && a.window > 0 ? place - a.window + 1 : 0;
            all_hi = min(all_hi, hi_key[ct]), any_hi = max(any_hi, hi_key[ct]);
            any_lo = min(any_lo, lo_key[ct]), all_lo = max(all_lo, lo_key[ct]);
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            all_hi = min(all_hi, __shfl_xor(all_hi, d)), any_hi = max(any_hi, __shfl_xor(any_hi, d));
            any_lo = min(any_lo, __shfl_xor(any_lo, d)), all_lo = max(all_lo, __shfl_xor(all_lo, d));
        }
        all_hi = __builtin_amdgcn_readfirstlane(all_hi), any_hi = __builtin_amdgcn_readfirstlane(any_hi);
        any_lo = __builtin_amdgcn_readfirstlane(any_lo), all_lo = __builtin_amdgcn_readfirstlane(all_lo);
        // the split's steps, cut to the keys that some column sees
        int s0 = max(split * per, max(any_lo, 0) >> 6);
        int s1 = min(min((split + 1) * per, steps), (max(any_hi, 0) + 63) >> 6);
        if (r0 >= rows) s1 = s0;
        const int stride = shared ? 4 : 1;
        if (shared) s0 += wave;

        f32x4 acc[CT][2 * NB] = {};
        float m[CT], l[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) m[ct] = -INFINITY, l[ct] = 0.0f;
        KvStep<D, INT4> cur, nxt;
        if (s0 < s1) ka_load<D, INT4>(cur, a, table, head, 64 * s0, kv, lane);
        for (int s = s0; s < s1; s += stride) {
            if (s + stride < s1) ka_load<D, INT4>(nxt, a, table, head, 64 * (s + stride), kv, lane);
            const int key0 = 64 * s;
            // scores of keys 16 b + 4 t + i
            float p[CT][16];
#pragma unroll
            for (int g = 0; g < (INT4 ? NG : 1); ++g) {
                f32x4 sc[CT][4] = {};
#pragma unroll
                for (int k = (INT4 ? 2 * g : 0); k < (INT4 ? 2 * g + 2 : KS); ++k) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const bf16x8 kk = ka_k_operand<INT4>(cur.k[t][k], INT4 ? 0.0f : cur.ks[t]);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
                            sc[ct][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[ct][k], sc[ct][t], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    float x[16];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[4 * t + i] = sc[ct][t][i];
                    if constexpr (!INT4) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[ct][i] = x[i];
                    } else if (g == 0) {
                        ka_scale_keys(p[ct], x, cur.ks[0]);
                    } else {
                        ka_fma_keys(p[ct], x, cur.ks[g]);
                    }
                }
            }
            const bool mask = key0 + 64 > all_hi || key0 < all_lo || __any(!cur.ok);
            if (mask) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = key0 + 16 * b + i;
                        const bool see = cur.ok && key < hi_key[ct] && key >= lo_key[ct];
                        p[ct][i] = see ? p[ct][i] : -INFINITY;
                    }
            }
            // running maximum; probabilities
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float mx = p[ct][0];
#pragma unroll
                for (int i = 1; i < 16; ++i) mx = fmaxf(mx, p[ct][i]);
                mx = fmaxf(ka_max_parts(mx), m[ct]);
                if (__any(mx > m[ct])) {
                    const float f = m[ct] == mx ? 1.0f : __builtin_amdgcn_exp2f((m[ct] - mx) * c2);
                    l[ct] *= f;
#pragma unroll
                    for (int n = 0; n < 2 * NB; ++n) acc[ct][n] *= f;
                    m[ct] = mx;
                }
                const float base = mx == -INFINITY ? 0.0f : -mx * c2;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    p[ct][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[ct][i], c2, base));
                    sum += p[ct][i];
                }
                l[ct] += sum;
            }
            // O^T += V^T P^T
            constexpr int PG = INT4 ? NG : 1;
#pragma unroll
            for (int g = 0; g < PG; ++g) {
                bf16x8 pb[CT][2];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    float x[16];
                    if constexpr (INT4) {
                        ka_scale_keys(x, p[ct], cur.vs[g]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = p[ct][i];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pb[ct][h] = __builtin_bit_cast(bf16x8, (u32x4){ka_pack2(x[8 * h], x[8 * h + 1]), ka_pack2(x[8 * h + 2], x[8 * h + 3]),
                                                                       ka_pack2(x[8 * h + 4], x[8 * h + 5]), ka_pack2(x[8 * h + 6], x[8 * h + 7])});
                }
#pragma unroll
                for (int n = g * (NB / PG); n < (g + 1) * (NB / PG); ++n) {
                    bf16x8 lo, hi;
                    ka_v_operands<INT4, 0>(cur.v[n][0], cur.v[n][1], INT4 ? 0.0f : cur.vs[n % NG], lo, hi);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        acc[ct][2 * n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, pb[ct][0], acc[ct][2 * n], 0, 0, 0);
                        acc[ct][2 * n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, pb[ct][0], acc[ct][2 * n + 1], 0, 0, 0);
                    }
                    ka_v_operands<INT4, 1>(cur.v[n][2], cur.v[n][3], INT4 ? 0.0f : cur.vs[n % NG], lo, hi);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        acc[ct][2 * n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, pb[ct][1], acc[ct][2 * n], 0, 0, 0);
                        acc[ct][2 * n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, pb[ct][1], acc[ct][2 * n + 1], 0, 0, 0);
                    }
                }
            }
            cur = nxt;
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) l[ct] = ka_sum_parts(l[ct]);

        if (shared) {
            // the waves' parts, in wave order, into om
            if (b == 0) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) mm[wave][16 * ct + j] = m[ct], ll[wave][16 * ct + j] = l[ct];
            }
            __syncthreads();
            float f[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int r = 16 * ct + j;
                const float mx = fmaxf(fmaxf(mm[0][r], mm[1][r]), fmaxf(mm[2][r], mm[3][r]));
                f[ct] = m[ct] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m[ct] - mx) * c2);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (wave == w) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int n = 0; n < 2 * NB; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float &o = om[16 * ct + j][16 * n + 4 * b + i];
                                o = (w == 0 ? 0.0f : o) + acc[ct][n][i] * f[ct];
                            }
                }
                __syncthreads();
            }
            const int nr = (int)rows;
            for (int e = tid; e < nr * (D / 4); e += 256) {
                const int r = e / (D / 4), c = 4 * (e % (D / 4));
                const float mx = fmaxf(fmaxf(mm[0][r], mm[1][r]), fmaxf(mm[2][r], mm[3][r]));
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    sum += mm[w][r] == -INFINITY ? 0.0f : ll[w][r] * __builtin_amdgcn_exp2f((mm[w][r] - mx) * c2);
                const size_t row = (size_t)(qs + r / G) * a.heads_q + head * G + r % G;
                const float4 o = *reinterpret_cast<const float4 *>(&om[r][c]);
                if (a.splits > 1) {
                    const size_t part = (size_t)split * a.T * a.heads_q + row;
                    *reinterpret_cast<float4 *>(a.work + part * D + c) = o;
                    if (c == 0) {
                        float *ml = a.work + (size_t)a.splits * a.T * a.heads_q * D + 2 * part;
                        ml[0] = mx * a.scale, ml[1] = sum;
                    }
                } else {
                    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
                    *reinterpret_cast<uint2 *>(a.O + row * D + c) =
                        make_uint2(ka_pack2(o.x * inv, o.y * inv), ka_pack2(o.z * inv, o.w * inv));
                    if (c == 0 && a.lse)
                        a.lse[row] = sum == 0.0f ? -INFINITY : mx * a.scale + kLn2 * __builtin_amdgcn_logf(sum);
                }
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int64_t r = r0 + 16 * ct + j;
                if (r >= rows) continue;
                const size_t row = (size_t)(qs + (int)(r / G)) * a.heads_q + head * G + (int)(r % G);
                if (a.splits > 1) {
                    const size_t part = (size_t)split * a.T * a.heads_q + row;
#pragma unroll
                    for (int n = 0; n < 2 * NB; ++n)
                        *reinterpret_cast<float4 *>(a.work + part * D + 16 * n + 4 * b) =
                            make_float4(acc[ct][n][0], acc[ct][n][1], acc[ct][n][2], acc[ct][n][3]);
                    if (b == 0) {
                        float *ml = a.work + (size_t)a.splits * a.T * a.heads_q * D + 2 * part;
                        ml[0] = m[ct] * a.scale, ml[1] = l[ct];
                    }
                } else {
                    const float inv = l[ct] > 0.0f ? 1.0f / l[ct] : (l[ct] == 0.0f ? 0.0f : l[ct]);
#pragma unroll
                    for (int n = 0; n < 2 * NB; ++n)
                        *reinterpret_cast<uint2 *>(a.O + row * D + 16 * n + 4 * b) =
                            make_uint2(ka_pack2(acc[ct][n][0] * inv, acc[ct][n][1] * inv),
                                       ka_pack2(acc[ct][n][2] * inv, acc[ct][n][3] * inv));
                    if (b == 0 && a.lse)
                        a.lse[row] = l[ct] == 0.0f ? -INFINITY : m[ct] * a.scale + kLn2 * __builtin_amdgcn_logf(l[ct]);
                }
            }
        }
    }
}

// O = sum over the splits, in split order; one wave per row.
template <int D>
__global__ __launch_bounds__(256) void kv4_combine_kernel(KvArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t n = (int64_t)a.T * a.heads_q;
    // rows outside the sequences keep what they hold
    if (row >= n || row < (int64_t)a.q_start[0] * a.heads_q || row >= (int64_t)a.q_start[a.B] * a.heads_q) return;
    const float *ml = a.work + (size_t)a.splits * n * D;
    float mx = -INFINITY;
    for (int s = 0; s < a.splits; ++s) mx = fmaxf(mx, ml[2 * (s * n + row)]);
    float sum = 0.0f;
    constexpr int C = D / 64;
    float o[C] = {};
    for (int s = 0; s < a.splits; ++s) {
        const float ms = ml[2 * (s * n + row)];
        if (ms == -INFINITY) continue;
        const float f = __builtin_amdgcn_exp2f((ms - mx) * kLog2e);
        sum = __builtin_fmaf(ml[2 * (s * n + row) + 1], f, sum);
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = __builtin_fmaf(a.work[(s * n + row) * D + C * lane + c], f, o[c]);
    }
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
    if constexpr (C == 2) *reinterpret_cast<uint32_t *>(a.O + row * D + 2 * lane) = ka_pack2(o[0] * inv, o[1] * inv);
    else a.O[row * D + lane] = (uint16_t)ka_pack2(o[0] * inv, 0.0f);
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : mx + kLn2 * __builtin_amdgcn_logf(sum);
}

// Tiles of rows, rows per wave and splits of the keys, from the sizes and the
// caller's bounds.  Few rows: 16 per wave, shared by the block's waves.
struct KvPlan {
    int ct, q_tiles, splits;
};

KvPlan ka_plan(int B, int heads, int group, int max_q, int max_kv)
{
    KvPlan p;
    const int64_t rows = (int64_t)max_q * group;
    const int cus = device_cu_count();
    p.ct = rows <= 16 ? 1 : 2;
    const int block_rows = rows <= 16 * p.ct ? 16 * p.ct : 64 * p.ct;
    const int64_t tiles = (rows + block_rows - 1) / block_rows;
    const int64_t blocks = tiles * B * heads;
    // a split keeps at least eight steps of 64 keys (two per wave)
    const int64_t most = max_kv / 512;
    int64_t s = (2 * (int64_t)cus + blocks - 1) / blocks;
    s = s > most ? most : s;
    p.splits = (int)(s < 1 ? 1 : (s > 64 ? 64 : s));
    const int64_t cap = (int64_t)(1 << 24) / ((int64_t)B * heads * p.splits) + 1;    // grid; further tiles in a loop
    p.q_tiles = (int)(tiles > cap ? cap : tiles);
    return p;
}

}  // namespace

size_t kv4_attention_work_bytes(int T, int B, int heads_q, int heads, int dim, int max_q, int max_kv)
{
    const KvPlan p = ka_plan(B, heads, heads_q / heads, max_q, max_kv);
    return p.splits > 1 ? (size_t)p.splits * T * heads_q * (dim + 2) * sizeof(float) : 0;
}

hipError_t launch_kv4_attention(const Kv4View &c, const uint16_t *Q, int64_t ldq, const int32_t *table, int table_width,
                                const int32_t *q_start, const int32_t *kv_len, int B, int T, int heads_q, int max_q,
                                int max_kv, float scale, int causal, int window, uint16_t *O, float *lse, float *work,
                                hipStream_t stream)
{
    const KvPlan p = ka_plan(B, c.heads, heads_q / c.heads, max_q, max_kv);
    KvArgs a{};
    a.c = c, a.Q = Q, a.ldq = ldq, a.table = table, a.q_start = q_start, a.kv_len = kv_len, a.O = O, a.lse = lse;
    a.work = work, a.T = T, a.B = B, a.heads_q = heads_q, a.group = heads_q / c.heads, a.table_width = table_width;
    a.q_tiles = p.q_tiles, a.splits = p.splits, a.causal = causal, a.window = window, a.scale = scale;
    const dim3 grid((uint32_t)((int64_t)p.q_tiles * p.splits * B * c.heads));
#define KA_LAUNCH(D, I) \
    (p.ct == 1 ? kv4_attention_kernel<D, I, 1><<<grid, 256, 0, stream>>>(a) : kv4_attention_kernel<D, I, 2><<<grid, 256, 0, stream>>>(a))
    if (c.int4 && c.dim == 64) KA_LAUNCH(64, true);
    else if (c.int4) KA_LAUNCH(128, true);
    else if (c.dim == 64) KA_LAUNCH(64, false);
    else KA_LAUNCH(128, false);
#undef KA_LAUNCH
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const dim3 cgrid((uint32_t)(((int64_t)T * heads_q + 3) / 4));
    if (c.dim == 64) kv4_combine_kernel<64><<<cgrid, 256, 0, stream>>>(a);
    else kv4_combine_kernel<128><<<cgrid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace svdq
