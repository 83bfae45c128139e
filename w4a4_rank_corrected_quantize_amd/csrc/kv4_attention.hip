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
// and rescaling are per lane.  A step is 64 keys, four runs of 16; lane part b
// = lane / 16 gets the scores of tokens 4 b .. 4 b + 3 of every run, and these
// are the tokens that it reads of V, so the probabilities go from one product
// to the next in registers.  The page layout (kv4.h) has every run in operand
// order: a lane's part is 16 (D = 64: 8) consecutive bytes, a wave's one run
// (in plain token order, a lane per token, the loads took four times the L1's
// cycles).
//
// INT4 scales (fp32) belong to a key and a 64-channel group: lane (b, j) holds
// the scale of token 4 b + j % 4 of run j / 4 and the lanes of part b multiply
// with a broadcast from it (DPP).  K's multiply the group's score sums, V's the
// probabilities before they are rounded to bf16.  MXFP4 scales enter the fp4 ->
// bf16 conversion itself.
//
// Rounding choices: p (INT4: p times V's scale) is rounded to bf16 for the
// second product (at most 2^-8 relative, as the output's own type rounds);
// the sum of p is taken of the unrounded values.
//
// Rows are packed: the G = heads_q / heads query heads that share a key head
// and the sequence's new tokens form one list, row = token G + head, so single
// tokens of grouped heads fill the 16 columns of a product.
//   Up to 16 rows (decoding): a block takes 16 rows, its four waves every
//   fourth step each, codes straight from memory to registers one step ahead;
//   the waves' sums are added in LDS in wave order.
//   More: a block takes 128 rows, 32 per wave.  The conversion of a step's codes
//   is shared: each wave converts a quarter into LDS and all read the whole.
// The keys are split over blocks where rows alone do not fill the chip; the
// splits' sums then go to the workspace and a second kernel adds them in split
// order.
//
// What bounds it, and what it measured (both kernels, in a captured graph):
//   32 x 4097 .. 16384 keys, 32 heads over 8 of 128, one token each: MXFP4 76 us
//   for 335 MB = 4.4 TB/s (a large copy: 5.4 TB/s), INT4 81 us for 355 MB.  Bound
//   by HBM; the first form, with codes in token order and block tables in vector
//   loads, took 109 us (MXFP4).
//   4608 rows over 4608 keys, 24 heads: D = 128 MXFP4 290 us = 900 TFLOP/s,
//   INT4 375 us; D = 64 203 and 238 us; causal, 32 heads over 8 of 128: 190 and
//   237 us.  Bound by instruction issue: a step of a
//   wave issues 64 (32) matrix instructions, 32 exponentials and about 210
//   other vector instructions, which the products do not hide (a matrix
//   instruction holds the port for half of its time), and by the 864 tiles over
//   512 places.  Before scores, exponentials and conversions were interleaved:
//   340 us; before the shared conversion: 445 us.
//   One token over 1000 keys, 32 heads over 8: 7.7 + 2.6 us, latencies of the
//   dependent loads (lengths, table, codes) and of the second launch.
//   8 sequences of 1 .. 700 rows over up to 6000 keys, 16 heads over 4 of 64,
//   INT4, causal: 103 us = 288 TFLOP/s; some 780 pieces of about 20 steps over
//   512 places, two rounds.
// Not kept: 48 rows per wave and three waves per SIMD (spills), 64 rows and one
// wave per SIMD (443 us: nothing beside a wave's waits), a branch
// around the rescaling per column (copies of the sums), ordering hints instead
// of fences (the compiler regrouped the pieces), several heads per block.
#include "kv4.h"
#include "kv4_plan.h"

namespace svdq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLazy = 8.0f;

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

// The same for a J known after unrolling.
__device__ __forceinline__ float ka_bcast(float x, int j)
{
    switch (j) {
    case 0: return ka_row_bcast<0>(x);
    case 1: return ka_row_bcast<1>(x);
    case 2: return ka_row_bcast<2>(x);
    case 3: return ka_row_bcast<3>(x);
    case 4: return ka_row_bcast<4>(x);
    case 5: return ka_row_bcast<5>(x);
    case 6: return ka_row_bcast<6>(x);
    case 7: return ka_row_bcast<7>(x);
    case 8: return ka_row_bcast<8>(x);
    case 9: return ka_row_bcast<9>(x);
    case 10: return ka_row_bcast<10>(x);
    case 11: return ka_row_bcast<11>(x);
    case 12: return ka_row_bcast<12>(x);
    case 13: return ka_row_bcast<13>(x);
    case 14: return ka_row_bcast<14>(x);
    default: return ka_row_bcast<15>(x);
    }
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
    int T, B, heads_q, group, table_width, q_tiles, splits, split_steps, causal, window, cus;
    float scale;
};

// One step's codes and scales in flight.
template <int D, bool INT4>
struct KvStep {
    static constexpr int KS = D / 32;             // 32-channel product steps = dwords of a lane's K part
    static constexpr int NB = D / 32;             // 32-channel blocks of V
    static constexpr int NG = INT4 ? D / 64 : D / 32;
    uint32_t k[4][KS], v[4][NB];                  // run t
    float ks[INT4 ? NG : 4];                      // INT4: of the lane's scale key; MXFP4: of the K row of run t
    float vs[NG];                                 // of the lane's scale key
    int valid;                                    // bit t: run t lies in a page of the cache
};

// The block tables and lengths are read through scalar loads: their addresses
// are uniform, and the count of vector loads in flight stays that of the codes
// (a page number from a vector load made every step wait for the codes issued
// before it).
typedef const __attribute__((address_space(4))) int32_t ka_const_int;

// Pages of the four runs of a step; one where a page holds a whole step.
struct KvPages {
    int p[4];
};

__device__ __forceinline__ KvPages ka_pages(const KvArgs &a, ka_const_int *table, int key0, int kv_end)
{
    KvPages g;
    const int top = max(kv_end - 1, 0);                 // always an entry of the table
    g.p[0] = table[min(key0, top) >> a.c.page_shift];
    if (a.c.page_shift >= 6) {
        g.p[1] = g.p[2] = g.p[3] = g.p[0];
    } else {
#pragma unroll
        for (int t = 1; t < 4; ++t) g.p[t] = table[min(key0 + 16 * t, top) >> a.c.page_shift];
    }
    return g;
}

// The four runs' numbers in the cache, and which of them hold keys (bit t).
struct KvRuns {
    int64_t run[4];
    int valid;
};

__device__ __forceinline__ KvRuns ka_runs(const KvArgs &a, const KvPages &pg, int head, int key0, int kv_end)
{
    KvRuns r;
    const int left = kv_end - key0;
    const int in = left > 48 ? 15 : (left > 32 ? 7 : (left > 16 ? 3 : (left > 0 ? 1 : 0)));
    const int mask = (1 << a.c.page_shift) - 1, rs = a.c.page_shift - 4;
    const int page = (uint32_t)pg.p[0] < (uint32_t)a.c.pages ? pg.p[0] : 0;      // not used then; page 0 exists
    const int ok0 = (uint32_t)pg.p[0] < (uint32_t)a.c.pages ? 15 : 0;
    r.run[0] = (((int64_t)page * a.c.heads + head) << rs) + ((key0 & mask) >> 4);
    if (a.c.page_shift >= 6) {
        r.run[1] = r.run[0] + 1, r.run[2] = r.run[0] + 2, r.run[3] = r.run[0] + 3;
        r.valid = ok0 & in;
    } else {
        int ok = ok0 & 1;
#pragma unroll
        for (int t = 1; t < 4; ++t) {
            const bool good = (uint32_t)pg.p[t] < (uint32_t)a.c.pages;
            r.run[t] = (((int64_t)(good ? pg.p[t] : 0) * a.c.heads + head) << rs) + (((key0 + 16 * t) & mask) >> 4);
            ok |= good ? 1 << t : 0;
        }
        r.valid = ok & in;
    }
    return r;
}

// Run t (values, not a choice between addresses, which would put the runs in
// memory).
__device__ __forceinline__ int64_t ka_pick(const KvRuns &r, int t)
{
    const int64_t a = r.run[0], b = r.run[1], c = r.run[2], d = r.run[3];
    const int64_t lo = t & 1 ? b : a, hi = t & 1 ? d : c;
    return t & 2 ? hi : lo;
}

// The keys that a block's rows see: steps s0 .. s1 - 1, keys lo .. hi - 1.
struct KvRange {
    int s0, s1, lo, hi;
};

// All ones where bit 0 of `valid` is set and the key lies in the range, else 0.
// The scale of a V place that no row sees becomes 0 with it (the place may hold
// anything, and 0 times that need not be 0; what append wrote is finite); as a
// select, the compiler loads under a condition.
__device__ __forceinline__ uint32_t ka_in_mask(int valid, int key, const KvRange &g)
{
    return (uint32_t)(-(valid & 1) & ((key - g.hi) >> 31) & ((g.lo - 1 - key) >> 31));
}

template <int D, bool INT4>
__device__ __forceinline__ void ka_load(KvStep<D, INT4> &st, const KvArgs &a, const KvPages &pg, int head, int key0,
                                        const KvRange &g, int lane)
{
    constexpr int NG = KvStep<D, INT4>::NG;
    const int j = lane & 15, b = lane >> 4;
    const KvRuns r = ka_runs(a, pg, head, key0, g.hi);
    st.valid = r.valid;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint8_t *kp = a.c.k_codes + r.run[t] * (8 * D) + (D / 8) * lane;
        const uint8_t *vp = a.c.v_codes + r.run[t] * (8 * D) + (D / 8) * lane;
        if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4 *>(kp), w = *reinterpret_cast<const uint4 *>(vp);
            st.k[t][0] = u.x, st.k[t][1] = u.y, st.k[t][2] = u.z, st.k[t][3] = u.w;
            st.v[t][0] = w.x, st.v[t][1] = w.y, st.v[t][2] = w.z, st.v[t][3] = w.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(kp), w = *reinterpret_cast<const uint2 *>(vp);
            st.k[t][0] = u.x, st.k[t][1] = u.y;
            st.v[t][0] = w.x, st.v[t][1] = w.y;
        }
    }
    // the lane's scale key: token 4 b + j % 4 of run j / 4
    const int sr = j >> 2, tok = 4 * b + (j & 3);
    const int64_t mine = ka_pick(r, sr);
    const uint32_t in = ka_in_mask(st.valid >> sr, key0 + 16 * sr + tok, g);
    const int64_t so = mine * (16 * NG) + tok;
    if constexpr (INT4) {
        const float *ks = (const float *)a.c.k_scales + so, *vs = (const float *)a.c.v_scales + so;
#pragma unroll
        for (int i = 0; i < NG; ++i) st.ks[i] = ks[16 * i];
#pragma unroll
        for (int i = 0; i < NG; ++i) st.vs[i] = bits_f32(f32_bits(vs[16 * i]) & in);
    } else {
        const int blk = D == 128 ? b : b >> 1;    // the 32-channel block of the lane's K part
#pragma unroll
        for (int t = 0; t < 4; ++t)
            st.ks[t] = bits_f32((uint32_t)((const uint8_t *)a.c.k_scales)[r.run[t] * (16 * NG) + 16 * blk + j] << 23);
        const uint8_t *vs = (const uint8_t *)a.c.v_scales + so;
#pragma unroll
        for (int i = 0; i < NG; ++i) st.vs[i] = bits_f32(((uint32_t)vs[16 * i] << 23) & in);
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

// Operands of 8 keys (the dwords of two runs) for the low- and the high-nibble
// channel.  S: runs 0 and 1 or 2 and 3 (for the scales).
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

// A second register with the same value: the compiler shares a lane's
// broadcast among its uses and folds it (DPP) only into a single one.
__device__ __forceinline__ float ka_copy(float x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// o[4 t + i] = / += x[4 t + i] times the scale of token i of the lane's part of run t.
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

// First key that a row at this place sees.
__device__ __forceinline__ int ka_window(const KvArgs &a, int place)
{
    return a.causal && a.window > 0 ? (int)max((int64_t)place - a.window + 1, (int64_t)0) : 0;
}

// A wave's rows: 16 CT query rows of one key head, column 16 ct + j each.
template <int D, int CT>
struct KvRows {
    bf16x8 q[CT][D / 32];
    f32x4 acc[CT][D / 16];                        // O^T, tile (block n, half h) at 2 n + h
    float m[CT], l[CT];                           // running maximum; the lane part's share of the sum
    int hi_key[CT], lo_key[CT];                   // the columns' keys: lo <= key < hi
    int all_hi, all_lo;                           // over the columns: the least hi, the greatest lo
};

template <int D, bool INT4, int CT>
__device__ __forceinline__ void ka_rows(KvRows<D, CT> &w, const KvArgs &a, int head, int qs, int qn, int kv, int64_t r0,
                                        int64_t rows, int lane)
{
    const int j = lane & 15, b = lane >> 4, G = a.group;
    w.all_hi = kv, w.all_lo = 0;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int64_t r = min(r0 + 16 * ct + j, rows - 1);      // rows past the last repeat it, never stored
        const int tok = (int)(r / G), hd = head * G + (int)(r % G);
        const uint16_t *qp = a.Q + (qs + tok) * a.ldq + (int64_t)hd * D;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            const int ch = INT4 ? 64 * (k >> 1) + 16 * b + 8 * (k & 1) : (D / 4) * b + 8 * k;
            w.q[ct][k] = *reinterpret_cast<const bf16x8 *>(qp + ch);
        }
        const int place = kv - qn + tok;
        w.hi_key[ct] = a.causal ? min(place + 1, kv) : kv;
        w.lo_key[ct] = ka_window(a, place);
        w.all_hi = min(w.all_hi, w.hi_key[ct]), w.all_lo = max(w.all_lo, w.lo_key[ct]);
        w.m[ct] = -INFINITY, w.l[ct] = 0.0f;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) w.acc[ct][n] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int d = 1; d < 16; d <<= 1)
        w.all_hi = min(w.all_hi, __shfl_xor(w.all_hi, d)), w.all_lo = max(w.all_lo, __shfl_xor(w.all_lo, d));
    w.all_hi = __builtin_amdgcn_readfirstlane(w.all_hi), w.all_lo = __builtin_amdgcn_readfirstlane(w.all_lo);
}

// Before a step's exponentials: scores (run t, token 4 b + i at 4 t + i) that a
// row does not see become -infinity, and the reference m moves where a score
// exceeds it by more than kLazy (seen in any lane): p is at most 2^kLazy then,
// and its relative rounding the same.
template <int D, int CT>
__device__ __forceinline__ void ka_reference(KvRows<D, CT> &w, float (&p)[CT][16], int key0, int valid, float c2, int b)
{
    if (key0 + 64 > w.all_hi || key0 < w.all_lo || valid != 15) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int key = key0 + 16 * (i >> 2) + 4 * b + (i & 3);
                const bool see = ((valid >> (i >> 2)) & 1) && key < w.hi_key[ct] && key >= w.lo_key[ct];
                p[ct][i] = see ? p[ct][i] : -INFINITY;
            }
    }
    float mx[CT];
    bool up = false;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        mx[ct] = p[ct][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx[ct] = fmaxf(mx[ct], p[ct][i]);
        up |= (mx[ct] - w.m[ct]) * c2 > kLazy;
    }
    if (__any(up)) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const float top = fmaxf(ka_max_parts(mx[ct]), w.m[ct]);
            const float f = w.m[ct] == top ? 1.0f : __builtin_amdgcn_exp2f((w.m[ct] - top) * c2);
            w.l[ct] *= f;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) w.acc[ct][n] *= f;
            w.m[ct] = top;
        }
    }
}

// Probabilities, and their sum.
template <int D, int CT>
__device__ __forceinline__ void ka_exponentials(KvRows<D, CT> &w, float (&p)[CT][16], float c2)
{
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const float base = w.m[ct] == -INFINITY ? 0.0f : -w.m[ct] * c2;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            p[ct][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[ct][i], c2, base));
            sum += p[ct][i];
        }
        w.l[ct] += sum;
    }
}

// Operands of the second product: keys of runs 2 h and 2 h + 1.
__device__ __forceinline__ void ka_p_operands(const float (&x)[16], bf16x8 (&pb)[2])
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
        pb[h] = __builtin_bit_cast(bf16x8, (u32x4){ka_pack2(x[8 * h], x[8 * h + 1]), ka_pack2(x[8 * h + 2], x[8 * h + 3]),
                                                   ka_pack2(x[8 * h + 4], x[8 * h + 5]), ka_pack2(x[8 * h + 6], x[8 * h + 7])});
}

// Scores of a step: k_op(t, k) gives K's operand of run t and product step k, ks
// the lane's INT4 scales.
template <int D, bool INT4, int CT, class KOp>
__device__ __forceinline__ void ka_scores(const KvRows<D, CT> &w, float (&p)[CT][16], const float *ks, KOp k_op)
{
    constexpr int KS = D / 32, NG = INT4 ? D / 64 : 1;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        f32x4 sc[CT][4] = {};
#pragma unroll
        for (int k = g * (KS / NG); k < (g + 1) * (KS / NG); ++k)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const bf16x8 kk = k_op(t, k);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    sc[ct][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, w.q[ct][k], sc[ct][t], 0, 0, 0);
            }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = sc[ct][i >> 2][i & 3];
            if constexpr (!INT4) {
#pragma unroll
                for (int i = 0; i < 16; ++i) p[ct][i] = x[i];
            } else if (g == 0) {
                ka_scale_keys(p[ct], x, ks[0]);
            } else {
                ka_fma_keys(p[ct], x, ks[g]);
            }
        }
    }
}

// Operands of the second product from the probabilities; vs: the lane's INT4
// scales, one set of operands per 64-channel group.
template <int D, bool INT4, int CT>
struct KvP {
    static constexpr int NG = INT4 ? D / 64 : 1;
    bf16x8 b[NG][CT][2];
};

template <int D, bool INT4, int CT>
__device__ __forceinline__ void ka_p(KvP<D, INT4, CT> &o, const float (&p)[CT][16], const float *vs)
{
#pragma unroll
    for (int g = 0; g < KvP<D, INT4, CT>::NG; ++g)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            if constexpr (INT4) {
                float x[16];
                ka_scale_keys(x, p[ct], vs[g]);
                ka_p_operands(x, o.b[g][ct]);
            } else {
                ka_p_operands(p[ct], o.b[g][ct]);
            }
        }
}

// O^T += V^T P^T: v_op(n, h, lo, hi) gives V's operands of block n and runs 2 h,
// 2 h + 1.
template <int D, bool INT4, int CT, class VOp>
__device__ __forceinline__ void ka_values(KvRows<D, CT> &w, const KvP<D, INT4, CT> &pb, VOp v_op)
{
    constexpr int NB = D / 32, NG = KvP<D, INT4, CT>::NG;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 lo, hi;
            v_op(n, h, lo, hi);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const bf16x8 b = pb.b[n / (NB / NG)][ct][h];
                w.acc[ct][2 * n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, b, w.acc[ct][2 * n], 0, 0, 0);
                w.acc[ct][2 * n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, b, w.acc[ct][2 * n + 1], 0, 0, 0);
            }
        }
}

// Few rows: the wave converts its own codes, steps s0, s0 + stride, .. < s1.
// Codes are one step ahead, their pages two; past the end the last run's page
// is looked up and nothing of it is used.
template <int D, bool INT4, int CT>
__device__ __forceinline__ void ka_walk(KvRows<D, CT> &w, const KvArgs &a, ka_const_int *table, int head, const KvRange &g,
                                        int s0, int stride, float c2, int lane)
{
    constexpr int NG = KvStep<D, INT4>::NG;
    const int s1 = g.s1;
    KvStep<D, INT4> x, y;
    if (s0 >= s1) return;
    auto compute = [&](const KvStep<D, INT4> &c, int s) {
        float p[CT][16];
        KvP<D, INT4, CT> pb;
        ka_scores<D, INT4, CT>(w, p, c.ks, [&](int t, int k) { return ka_k_operand<INT4>(c.k[t][k], INT4 ? 0.0f : c.ks[t]); });
        ka_reference<D, CT>(w, p, 64 * s, c.valid, c2, lane >> 4);
        ka_exponentials<D, CT>(w, p, c2);
        ka_p<D, INT4, CT>(pb, p, c.vs);
        ka_values<D, INT4, CT>(w, pb, [&](int n, int h, bf16x8 &lo, bf16x8 &hi) {
            const float vs = INT4 ? 0.0f : c.vs[n % NG];
            if (h == 0) ka_v_operands<INT4, 0>(c.v[0][n], c.v[1][n], vs, lo, hi);
            else ka_v_operands<INT4, 1>(c.v[2][n], c.v[3][n], vs, lo, hi);
        });
    };
    ka_load<D, INT4>(x, a, ka_pages(a, table, 64 * s0, g.hi), head, 64 * s0, g, lane);
    KvPages pages = ka_pages(a, table, 64 * (s0 + stride), g.hi);
    for (int s = s0;; s += 2 * stride) {
        ka_load<D, INT4>(y, a, pages, head, 64 * (s + stride), g, lane);
        pages = ka_pages(a, table, 64 * (s + 2 * stride), g.hi);
        compute(x, s);
        if (s + stride >= s1) break;
        ka_load<D, INT4>(x, a, pages, head, 64 * (s + 2 * stride), g, lane);
        pages = ka_pages(a, table, 64 * (s + 3 * stride), g.hi);
        compute(y, s + stride);
        if (s + 2 * stride >= s1) break;
    }
}

// Many rows: the block's four waves convert a step's codes together, a quarter
// each, into LDS (operand order, 16 bytes per lane: no bank conflicts), and
// every wave multiplies the whole step.
//
// The loop is skewed so that the matrix cores have work during the softmax: an
// iteration computes the scores of step s + 1 between the exponentials of step
// s, then the second product of step s between the conversions of K of step s
// + 2 and V of step s + 1.  K and V have two stages each; what an iteration
// writes was last read in the iteration before.
template <int D, bool INT4>
struct KvShareK {
    uint32_t k[D / 32];                           // run `wave`
    float ks;                                     // MXFP4: of the K row
    float iks[2];                                 // INT4: the lane's scales, as in KvStep
    int valid;
};

template <int D, bool INT4>
struct KvShareV {
    uint32_t v[2][D / 64];                        // runs 2 (wave / 2) and + 1, blocks D / 64 (wave % 2) ..
    float vq[D / 64];                             // MXFP4: of token 4 b + j % 4 of run 2 (wave / 2) + (j / 4) % 2
    float ivs[2];                                 // INT4: the lane's scales
};

template <int D, bool INT4>
__device__ __forceinline__ void ka_share_load_k(KvShareK<D, INT4> &st, const KvArgs &a, const KvRuns &r, int wave, int lane)
{
    constexpr int NG = INT4 ? D / 64 : D / 32;
    const int j = lane & 15, b = lane >> 4;
    st.valid = r.valid;
    const int64_t rk = ka_pick(r, wave);
    const uint8_t *kp = a.c.k_codes + rk * (8 * D) + (D / 8) * lane;
    if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4 *>(kp);
        st.k[0] = u.x, st.k[1] = u.y, st.k[2] = u.z, st.k[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(kp);
        st.k[0] = u.x, st.k[1] = u.y;
    }
    if constexpr (INT4) {
        const int sr = j >> 2, tok = 4 * b + (j & 3);
        const int64_t mine = ka_pick(r, sr);
        const float *ks = (const float *)a.c.k_scales + mine * (16 * NG) + tok;
#pragma unroll
        for (int g = 0; g < NG; ++g) st.iks[g] = ks[16 * g];
    } else {
        const int blk = D == 128 ? b : b >> 1;
        st.ks = bits_f32((uint32_t)((const uint8_t *)a.c.k_scales)[rk * (16 * NG) + 16 * blk + j] << 23);
    }
}

template <int D, bool INT4>
__device__ __forceinline__ void ka_share_load_v(KvShareV<D, INT4> &st, const KvArgs &a, const KvRuns &r, int key0,
                                                const KvRange &g, int wave, int lane)
{
    constexpr int NB = D / 32, NG = INT4 ? D / 64 : D / 32;
    const int j = lane & 15, b = lane >> 4, s2 = wave >> 1;
    const int64_t rv0 = ka_pick(r, 2 * s2), rv1 = ka_pick(r, 2 * s2 + 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint8_t *vp = a.c.v_codes + (i ? rv1 : rv0) * (8 * D) + (D / 8) * lane + 2 * NB * (wave & 1);
        if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2 *>(vp);
            st.v[i][0] = u.x, st.v[i][1] = u.y;
        } else {
            st.v[i][0] = *reinterpret_cast<const uint32_t *>(vp);
        }
    }
    if constexpr (INT4) {
        const int sr = j >> 2, tok = 4 * b + (j & 3);
        const int64_t mine = ka_pick(r, sr);
        const uint32_t in = ka_in_mask(r.valid >> sr, key0 + 16 * sr + tok, g);
        const float *vs = (const float *)a.c.v_scales + mine * (16 * NG) + tok;
#pragma unroll
        for (int i = 0; i < NG; ++i) st.ivs[i] = bits_f32(f32_bits(vs[16 * i]) & in);
    } else {
        const int sr = (j >> 2) & 1, tok = 4 * b + (j & 3);
        const uint32_t in = ka_in_mask(r.valid >> (2 * s2 + sr), key0 + 16 * (2 * s2 + sr) + tok, g);
        const uint8_t *vs = (const uint8_t *)a.c.v_scales + (sr ? rv1 : rv0) * (16 * NG) + tok;
#pragma unroll
        for (int n = 0; n < NB / 2; ++n)
            st.vq[n] = bits_f32(((uint32_t)vs[16 * (n + NB / 2 * (wave & 1))] << 23) & in);
    }
}

// Product step k of the wave's run.
template <int D, bool INT4>
__device__ __forceinline__ void ka_share_write_k(const KvShareK<D, INT4> &st, uint8_t *stage, int k, int wave, int lane)
{
    *reinterpret_cast<bf16x8 *>(stage + 1024 * (D / 32 * wave + k) + 16 * lane) = ka_k_operand<INT4>(st.k[k], INT4 ? 0.0f : st.ks);
}

// The wave's n-th block.
template <int D, bool INT4>
__device__ __forceinline__ void ka_share_write_v(const KvShareV<D, INT4> &st, uint8_t *stage, int n, int wave, int lane)
{
    constexpr int NB = D / 32;
    uint8_t *vb = stage + 2048 * (NB * (wave >> 1) + NB / 2 * (wave & 1) + n) + 16 * lane;
    bf16x8 lo, hi;
    ka_v_operands<INT4, 0>(st.v[0][n], st.v[1][n], INT4 ? 0.0f : st.vq[n], lo, hi);
    *reinterpret_cast<bf16x8 *>(vb) = lo;
    *reinterpret_cast<bf16x8 *>(vb + 1024) = hi;
}

typedef __attribute__((address_space(3))) uint8_t ka_lds_u8;
typedef const __attribute__((address_space(3))) bf16x8 ka_lds_bf16x8;

__device__ __forceinline__ bf16x8 ka_lds_read(uint32_t base, int off) { return *(ka_lds_bf16x8 *)(uintptr_t)(base + off); }

// Half e % 2 (low, high channel) of operand pair e / 2 of the second product.
template <int NB, int N>
__device__ __forceinline__ void ka_v_read(bf16x8 (&vf)[N][2], uint32_t base, int e)
{
    const int i = e >> 1;
    vf[i][e & 1] = ka_lds_read(base, 2048 * (NB * (i & 1) + (i >> 1)) + 1024 * (e & 1));
}

// Scores e, e + 1 (of column tile e / 16) to probabilities, their sum, and
// their place in the second product's operands.
template <int D, bool INT4, int CT>
__device__ __forceinline__ void ka_exp_pair(KvP<D, INT4, CT> &pb, const float (&p)[CT][16], float (&sum)[CT],
                                            const float (&base)[CT], float c2, const float (&vs)[CT][2], int e)
{
    const int ct = e >> 4, i = e & 15;
    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(p[ct][i], c2, base[ct]));
    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(p[ct][i + 1], c2, base[ct]));
    sum[ct] += x;
    sum[ct] += y;
#pragma unroll
    for (int g = 0; g < KvP<D, INT4, CT>::NG; ++g) {
        uint32_t u;
        if constexpr (INT4) u = ka_pack2(x * ka_bcast(vs[ct][g], i), y * ka_bcast(vs[ct][g], i + 1));
        else u = ka_pack2(x, y);
        u32x4 q = __builtin_bit_cast(u32x4, pb.b[g][ct][i >> 3]);
        q[(i & 7) >> 1] = u;
        pb.b[g][ct][i >> 3] = __builtin_bit_cast(bf16x8, q);
    }
}

// A group's sums into the scores.
template <bool INT4, int CT>
__device__ __forceinline__ void ka_take_scores(float (&p)[CT][16], const f32x4 (&sc)[CT][4], const float *ks, int g)
{
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = sc[ct][i >> 2][i & 3];
        if constexpr (!INT4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[ct][i] = x[i];
        } else if (g == 0) {
            ka_scale_keys(p[ct], x, ka_copy(ks[0]));
        } else {
            ka_fma_keys(p[ct], x, ks[g]);
        }
        if constexpr (INT4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+v"(p[ct][i]));
        }
    }
}

// Bytes of one stage of K or of V.
constexpr int ka_stage(int D) { return 128 * D; }

template <int D, bool INT4, int CT>
__device__ __forceinline__ void ka_walk_shared(KvRows<D, CT> &w, uint8_t *lds, const KvArgs &a, ka_const_int *table,
                                               int head, const KvRange &g, float c2, int wave, int lane)
{
    constexpr int KS = D / 32, NB = D / 32, STAGE = ka_stage(D), NG = INT4 ? D / 64 : 0, NS = INT4 ? NG : 1;
    constexpr int KO = 4 * KS, VO = 2 * NB;           // operands of the scores, operand pairs of the second product
    // INT4 heads of 128 need two sets of second operands and of sums: with the
    // scores next to the exponentials they spill (995 us against 476 at 4608 x
    // 4608, 24 heads), so the scores come after the second product there
    constexpr bool MIX = !(INT4 && D == 128);
    const int s0 = g.s0, s1 = g.s1;
    if (s0 >= s1) return;                             // the same for the whole block
    uint8_t *kb = lds, *vb = lds + 2 * STAGE;
    const uint32_t lb = (uint32_t)(uintptr_t)(const ka_lds_u8 *)lds + 16 * lane;
    auto runs = [&](int s, const KvPages &pg) { return ka_runs(a, pg, head, 64 * s, g.hi); };

    KvShareK<D, INT4> k2, k3;                         // K of step s + 2 (and s + 3, on its way)
    KvShareV<D, INT4> v1, v2;                         // V of step s + 1 (and s + 2)
    float ks1[2] = {}, vs0[2] = {};                   // INT4 scales: K of step s + 1, V of step s
    int valid1;                                       // of step s + 1
    float pa[CT][16], pc[CT][16];
    KvRuns r = runs(s0, ka_pages(a, table, 64 * s0, g.hi));
    ka_share_load_k<D, INT4>(k2, a, r, wave, lane);
    ka_share_load_v<D, INT4>(v1, a, r, 64 * s0, g, wave, lane);
    r = runs(s0 + 1, ka_pages(a, table, 64 * (s0 + 1), g.hi));
    ka_share_load_k<D, INT4>(k3, a, r, wave, lane);
    ka_share_load_v<D, INT4>(v2, a, r, 64 * (s0 + 1), g, wave, lane);
#pragma unroll
    for (int k = 0; k < KS; ++k) ka_share_write_k<D, INT4>(k2, kb, k, wave, lane), ka_share_write_k<D, INT4>(k3, kb + STAGE, k, wave, lane);
#pragma unroll
    for (int n = 0; n < NB / 2; ++n) ka_share_write_v<D, INT4>(v1, vb, n, wave, lane);
    valid1 = k3.valid;
    float ks0[2] = {};
#pragma unroll
    for (int i = 0; i < NG; ++i) ks0[i] = k2.iks[i], ks1[i] = k3.iks[i], vs0[i] = v1.ivs[i];
    const int valid0 = k2.valid;
    v1 = v2;
    r = runs(s0 + 2, ka_pages(a, table, 64 * (s0 + 2), g.hi));
    ka_share_load_k<D, INT4>(k2, a, r, wave, lane);
    KvPages pages = ka_pages(a, table, 64 * (s0 + 3), g.hi);
    __syncthreads();
    ka_scores<D, INT4, CT>(w, pa, ks0, [&](int t, int k) { return ka_lds_read(lb, 1024 * (KS * t + k)); });
    ka_reference<D, CT>(w, pa, 64 * s0, valid0, c2, lane >> 4);

    auto iteration = [&](int s, float (&cur)[CT][16], float (&nxt)[CT][16]) {
        const int x = (s - s0) & 1;
        uint8_t *k_now = kb + x * STAGE, *v_next = vb + (x ^ 1) * STAGE;
        const uint32_t lk = lb + (x ^ 1) * STAGE, lv = lb + (2 + x) * STAGE;
        __syncthreads();                              // K of step s + 1 and V of step s are written; the other stages free
        bf16x8 kf[KO], vf[VO][2];
        if (MIX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) kf[i] = ka_lds_read(lk, 1024 * (KS * (i & 3) + (i >> 2)));
        }
        // codes of the steps after
        ka_share_load_v<D, INT4>(v2, a, r, 64 * (s + 2), g, wave, lane);
        r = runs(s + 3, pages);
        ka_share_load_k<D, INT4>(k3, a, r, wave, lane);
        pages = ka_pages(a, table, 64 * (s + 4), g.hi);
        float base[CT], sum[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) base[ct] = w.m[ct] == -INFINITY ? 0.0f : -w.m[ct] * c2, sum[ct] = 0.0f;
        float vsc[CT][2] = {};
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int i = 0; i < NG; ++i) vsc[ct][i] = ka_copy(vs0[i]);
        __builtin_amdgcn_sched_barrier(0);
        KvP<D, INT4, CT> pb;
        // scores of step s + 1 (operand i: run i % 4, product step i / 4) and, in
        // between, the exponentials of step s: fenced pieces of CT products, an
        // operand read ahead, E exponentials and their bf16 pairs
        auto scores = [&] {
            constexpr int E = CT * 16 / KO;
            f32x4 sc[CT][4];
#pragma unroll
            for (int i = 0; i < KO; ++i) {
                if (i % (KO / NS) == 0) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int t = 0; t < 4; ++t) sc[ct][t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    sc[ct][i & 3] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[i], w.q[ct][i >> 2], sc[ct][i & 3], 0, 0, 0);
                if (i + 4 < KO) kf[i + 4] = ka_lds_read(lk, 1024 * (KS * (i & 3) + ((i + 4) >> 2)));
                else if (MIX) ka_v_read<NB>(vf, lv, i + 4 - KO);
                if (MIX) {
#pragma unroll
                    for (int e = E * i; e < E * (i + 1); e += 2) ka_exp_pair<D, INT4, CT>(pb, cur, sum, base, c2, vsc, e);
                }
                if ((i + 1) % (KO / NS) == 0) ka_take_scores<INT4, CT>(nxt, sc, ks1, (i + 1) / (KO / NS) - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (MIX) {
            scores();
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) ka_v_read<NB>(vf, lv, e);
#pragma unroll
            for (int e = 0; e < 16 * CT; e += 2) ka_exp_pair<D, INT4, CT>(pb, cur, sum, base, c2, vsc, e);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) w.l[ct] += sum[ct];
        // second product of step s (operand pair i: block i / 2, runs 2 (i % 2)
        // and + 1) and the conversions
#pragma unroll
        for (int i = 0; i < VO; ++i) {
            const int n = i >> 1, h = i & 1;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const bf16x8 p = pb.b[n / (NB / NS)][ct][h];
                w.acc[ct][2 * n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[i][0], p, w.acc[ct][2 * n], 0, 0, 0);
                w.acc[ct][2 * n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf[i][1], p, w.acc[ct][2 * n + 1], 0, 0, 0);
            }
            if (i + 2 < VO) ka_v_read<NB>(vf, lv, 2 * i + 4), ka_v_read<NB>(vf, lv, 2 * i + 5);
            if (i < KS) ka_share_write_k<D, INT4>(k2, k_now, i, wave, lane);
            else if (i < KS + NB / 2) ka_share_write_v<D, INT4>(v1, v_next, i - KS, wave, lane);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (!MIX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) kf[i] = ka_lds_read(lk, 1024 * (KS * (i & 3) + (i >> 2)));
            scores();
        }
        if (s + 1 < s1) ka_reference<D, CT>(w, nxt, 64 * (s + 1), valid1, c2, lane >> 4);
        valid1 = k2.valid;
#pragma unroll
        for (int i = 0; i < NG; ++i) ks1[i] = k2.iks[i], vs0[i] = v1.ivs[i];
        k2 = k3, v1 = v2;
    };
    for (int s = s0;; s += 2) {
        iteration(s, pa, pc);
        if (s + 1 >= s1) break;
        iteration(s + 1, pc, pa);
        if (s + 2 >= s1) break;
    }
    __syncthreads();
}

__device__ __forceinline__ float ka_inverse(float sum) { return sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum); }

__device__ __forceinline__ float ka_lse(float mx, float sum, float scale)
{
    return sum == 0.0f ? -INFINITY : mx * scale + kLn2 * __builtin_amdgcn_logf(sum);
}

// The keys of a tile of rows and a split.
__device__ __forceinline__ KvRange ka_range(const KvArgs &a, int split, int qn, int kv, int64_t r0, int64_t r1)
{
    const int first = kv - qn + (int)(r0 / a.group), last = kv - qn + (int)((r1 - 1) / a.group);
    const int lo = ka_window(a, first);
    const int hi = a.causal ? max(min(last + 1, kv), 0) : kv;
    // the tile's steps in as many equal parts as it takes for none to be longer
    // than split_steps (at most `splits` parts: longer ones then)
    const int s0 = lo >> 6, s1 = (hi + 63) >> 6, steps = max(s1 - s0, 0);
    const int parts = min(a.splits, (steps + a.split_steps - 1) / a.split_steps);
    const int per = parts > 1 ? ((steps + parts - 1) / parts + 3) & ~3 : steps;        // a step per wave
    return {min(s0 + split * per, s1), split < parts ? min(s0 + (split + 1) * per, s1) : s0, lo, hi};
}

// One row's four channels c .. of a block's or a wave's sums.
template <int D>
__device__ __forceinline__ void ka_store(const KvArgs &a, int split, size_t row, int c, f32x4 o, float mx, float sum)
{
    if (a.splits > 1) {
        const size_t part = (size_t)split * a.T * a.heads_q + row;
        if (mx != -INFINITY) *reinterpret_cast<f32x4 *>(a.work + part * D + c) = o;      // else not read
        if (c == 0) {
            float *ml = a.work + (size_t)a.splits * a.T * a.heads_q * D + 2 * part;
            ml[0] = mx * a.scale, ml[1] = sum;
        }
    } else {
        o *= ka_inverse(sum);
        *reinterpret_cast<uint2 *>(a.O + row * D + c) = make_uint2(ka_pack2(o[0], o[1]), ka_pack2(o[2], o[3]));
        if (c == 0 && a.lse) a.lse[row] = ka_lse(mx, sum, a.scale);
    }
}

// 16 rows, shared by the block's waves, which take the steps in turn.
template <int D, bool INT4>
__device__ __forceinline__ void ka_few_rows(float *om, const KvArgs &a, ka_const_int *table, int split, int head, int qs,
                                            int qn, int kv, int64_t r0, int64_t rows, int wave, int lane)
{
    const int j = lane & 15, b = lane >> 4, G = a.group;
    float (*mm)[16] = reinterpret_cast<float (*)[16]>(om + 16 * (D + 4)), (*ll)[16] = mm + 4;
    const float c2 = a.scale * kLog2e;
    KvRows<D, 1> w;
    ka_rows<D, INT4, 1>(w, a, head, qs, qn, kv, r0, rows, lane);
    const KvRange g = ka_range(a, split, qn, kv, r0, min(r0 + 16, rows));
    ka_walk<D, INT4, 1>(w, a, table, head, g, g.s0 + wave, 4, c2, lane);
    // the waves' parts, in wave order, into om
    const float l = ka_sum_parts(w.l[0]);
    if (b == 0) mm[wave][j] = w.m[0], ll[wave][j] = l;
    __syncthreads();
    const float mw = fmaxf(fmaxf(mm[0][j], mm[1][j]), fmaxf(mm[2][j], mm[3][j]));
    const float f = w.m[0] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((w.m[0] - mw) * c2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (wave == q) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                f32x4 *o = reinterpret_cast<f32x4 *>(om + j * (D + 4) + 16 * n + 4 * b);
                const f32x4 v = w.acc[0][n] * f;
                *o = q == 0 ? v : *o + v;
            }
        }
        __syncthreads();
    }
    const int nr = (int)min((int64_t)16, rows - r0);
    for (int e = 64 * wave + lane; e < nr * (D / 4); e += 256) {
        const int r = e / (D / 4), c = 4 * (e % (D / 4));
        const float mx = fmaxf(fmaxf(mm[0][r], mm[1][r]), fmaxf(mm[2][r], mm[3][r]));
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sum += mm[q][r] == -INFINITY ? 0.0f : ll[q][r] * __builtin_amdgcn_exp2f((mm[q][r] - mx) * c2);
        const int64_t rr = r0 + r;
        const size_t row = (size_t)(qs + (int)(rr / G)) * a.heads_q + head * G + (int)(rr % G);
        ka_store<D>(a, split, row, c, *reinterpret_cast<const f32x4 *>(om + r * (D + 4) + c), mx, sum);
    }
    __syncthreads();
}

// 64 CT rows, 16 CT per wave.
template <int D, bool INT4, int CT>
__device__ __forceinline__ void ka_many_rows(uint8_t *lds, const KvArgs &a, ka_const_int *table, int split, int head,
                                             int qs, int qn, int kv, int64_t r0, int64_t rows, int wave, int lane)
{
    const int j = lane & 15, b = lane >> 4, G = a.group;
    KvRows<D, CT> w;
    ka_rows<D, INT4, CT>(w, a, head, qs, qn, kv, r0 + 16 * CT * wave, rows, lane);
    const KvRange g = ka_range(a, split, qn, kv, r0, min(r0 + 64 * CT, rows));
    // Two blocks share a compute unit, so two waves a SIMD.  Blocks go out one per
    // compute unit at first: every other round of them gets precedence, and its
    // waves' waits are filled by the other's instead of both waiting in step
    // (4608 x 4608, 24 heads: MXFP4 300 -> 288 us, D = 64 218 -> 208; INT4 414
    // -> 399, 277 -> 265; by wave slots, which mixes a block's waves, slower than
    // without).
    if ((blockIdx.x / (uint32_t)a.cus) & 1) __builtin_amdgcn_s_setprio(2);
    ka_walk_shared<D, INT4, CT>(w, lds, a, table, head, g, a.scale * kLog2e, wave, lane);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const float l = ka_sum_parts(w.l[ct]);
        const int64_t r = r0 + 16 * CT * wave + 16 * ct + j;
        if (r >= rows) continue;
        const size_t row = (size_t)(qs + (int)(r / G)) * a.heads_q + head * G + (int)(r % G);
#pragma unroll
        for (int n = 0; n < D / 16; ++n) ka_store<D>(a, split, row, 16 * n + 4 * b, w.acc[ct][n], w.m[ct], l);
    }
}

// CT > 0: blocks of 64 CT rows for the sequences of more than 16.  0: every list
// of rows is taken 16 at a time.
template <int D, bool INT4, int CT>
__global__ __launch_bounds__(256, 2) void kv4_attention_kernel(KvArgs a)
{
    constexpr int SUMS = 4 * (16 * (D + 4) + 8 * 16), STAGES = 4 * ka_stage(D);
    __shared__ __attribute__((aligned(16))) uint8_t lds[CT > 0 && STAGES > SUMS ? STAGES : SUMS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // workgroups go to the XCDs in turn: rotating each round of heads and
    // sequences by one spreads a long sequence's tiles and splits over all
    const int n = a.c.heads * a.B, round = blockIdx.x / n;
    const int item = (int)((blockIdx.x % n + (uint32_t)round) % n);
    const int head = item % a.c.heads, seq = item / a.c.heads;
    const int split = round % a.splits, qt0 = round / a.splits;
    const int qs = min(max(((ka_const_int *)a.q_start)[seq], 0), a.T);
    const int qn = min(max(((ka_const_int *)a.q_start)[seq + 1], qs), a.T) - qs;
    const int kv = min(max(((ka_const_int *)a.kv_len)[seq], 0), a.table_width << a.c.page_shift);
    ka_const_int *table = (ka_const_int *)a.table + (size_t)seq * a.table_width;
    const int64_t rows = (int64_t)qn * a.group;
    const int block_rows = CT == 0 || rows <= 16 ? 16 : 64 * CT;
    // the last tiles first: under a causal mask they are the longest
    for (int64_t qt = (rows + block_rows - 1) / block_rows - 1 - qt0; qt >= 0; qt -= a.q_tiles) {
        if (block_rows == 16) ka_few_rows<D, INT4>(reinterpret_cast<float *>(lds), a, table, split, head, qs, qn, kv, 16 * qt, rows, wave, lane);
        else if constexpr (CT > 0) ka_many_rows<D, INT4, CT>(lds, a, table, split, head, qs, qn, kv, 64 * CT * qt, rows, wave, lane);
    }
}

// O = sum over the splits; D / 4 lanes per row and P parts of a block, part p
// with the splits p, p + P, .., the parts added in order.  Every split of every
// row of a sequence has been written, the ones without keys as a maximum of
// -infinity alone.
template <int D, int P>
__global__ __launch_bounds__(256) void kv4_combine_kernel(KvArgs a)
{
    constexpr int L = D / 4, R = 256 / (L * P);
    __shared__ f32x4 os[P > 1 ? P : 1][P > 1 ? R * L : 1];
    __shared__ float2 mls[P > 1 ? P : 1][P > 1 ? R : 1];
    const int lane = threadIdx.x % L, r = threadIdx.x / L % R, p = threadIdx.x / (L * R);
    const int64_t row = (int64_t)blockIdx.x * R + r;
    const int c = 4 * lane;
    const int64_t n = (int64_t)a.T * a.heads_q;
    // rows outside the sequences keep what they hold
    const bool in = row < n && row >= (int64_t)a.q_start[0] * a.heads_q && row < (int64_t)a.q_start[a.B] * a.heads_q;
    if (P == 1 && !in) return;
    const int64_t at = in ? row : 0;
    const float2 *ml = reinterpret_cast<const float2 *>(a.work + (size_t)a.splits * n * D) + at;
    const float *part = a.work + at * D + c;
    float mx = -INFINITY, sum = 0.0f;
    f32x4 o = {};
#pragma unroll 4
    for (int s = p; s < a.splits; s += P) mx = fmaxf(mx, ml[s * n].x);
#pragma unroll 4
    for (int s = p; s < a.splits; s += P) {
        const float2 v = ml[s * n];
        const bool none = v.x == -INFINITY;              // its sums are not written: any valid address, and 0
        const float f = none ? 0.0f : __builtin_amdgcn_exp2f((v.x - mx) * kLog2e);
        sum = __builtin_fmaf(v.y, f, sum);
        const f32x4 x = *reinterpret_cast<const f32x4 *>(part + (none ? 0 : s) * n * D);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = none ? o[i] : __builtin_fmaf(x[i], f, o[i]);
    }
    if constexpr (P > 1) {
        os[p][r * L + lane] = o;
        if (lane == 0) mls[p][r] = make_float2(mx, sum);
        __syncthreads();
        if (p > 0 || !in) return;
#pragma unroll
        for (int q = 1; q < P; ++q) mx = fmaxf(mx, mls[q][r].x);
        o = (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const float2 v = mls[q][r];
            const float f = v.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((v.x - mx) * kLog2e);
            sum = __builtin_fmaf(v.y, f, sum);
            o += os[q][r * L + lane] * f;
        }
    }
    o *= ka_inverse(sum);
    *reinterpret_cast<uint2 *>(a.O + row * D + c) = make_uint2(ka_pack2(o[0], o[1]), ka_pack2(o[2], o[3]));
    if (c == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : mx + kLn2 * __builtin_amdgcn_logf(sum);
}

}  // namespace

size_t kv4_attention_work_bytes(int T, int B, int heads_q, int heads, int dim, int max_q, int max_kv)
{
    const KvPlan p = kv4_plan(T, B, heads, heads_q / heads, max_q, max_kv, device_cu_count());
    return p.splits > 1 ? (size_t)p.splits * T * heads_q * (dim + 2) * sizeof(float) : 0;
}

hipError_t launch_kv4_attention(const Kv4View &c, const uint16_t *Q, int64_t ldq, const int32_t *table, int table_width,
                                const int32_t *q_start, const int32_t *kv_len, int B, int T, int heads_q, int max_q,
                                int max_kv, float scale, int causal, int window, uint16_t *O, float *lse, float *work,
                                hipStream_t stream)
{
    const int cus = device_cu_count();
    const KvPlan p = kv4_plan(T, B, c.heads, heads_q / c.heads, max_q, max_kv, cus);
    KvArgs a{};
    a.c = c, a.Q = Q, a.ldq = ldq, a.table = table, a.q_start = q_start, a.kv_len = kv_len, a.O = O, a.lse = lse;
    a.work = work, a.T = T, a.B = B, a.heads_q = heads_q, a.group = heads_q / c.heads, a.table_width = table_width;
    a.q_tiles = p.q_tiles, a.splits = p.splits, a.split_steps = p.split_steps, a.causal = causal, a.window = window, a.scale = scale;
    a.cus = cus;
    const dim3 grid((uint32_t)kv4_blocks(p, B, c.heads));
#define KA_LAUNCH(D, I) \
    (p.many ? kv4_attention_kernel<D, I, kKv4ManyTiles><<<grid, 256, 0, stream>>>(a) \
            : kv4_attention_kernel<D, I, 0><<<grid, 256, 0, stream>>>(a))
    if (c.int4 && c.dim == 64) KA_LAUNCH(64, true);
    else if (c.int4) KA_LAUNCH(128, true);
    else if (c.dim == 64) KA_LAUNCH(64, false);
    else KA_LAUNCH(128, false);
#undef KA_LAUNCH
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t n = (int64_t)T * heads_q;
#define KA_COMBINE(D, P) \
    kv4_combine_kernel<D, P><<<(uint32_t)((n * (D / 4 * P) + 255) / 256), 256, 0, stream>>>(a)
    if (p.splits <= 4) c.dim == 64 ? KA_COMBINE(64, 1) : KA_COMBINE(128, 1);
    else c.dim == 64 ? KA_COMBINE(64, 8) : KA_COMBINE(128, 8);
#undef KA_COMBINE
    return hipGetLastError();
}

}  // namespace svdq
