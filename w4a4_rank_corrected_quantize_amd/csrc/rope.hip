// rope.hip -- rotary positions with several axes: their tables, and the norm
// and rotation of query and key heads, on their own or on the way into the
// 4-bit cache.
//
//   angle_tp = pos_t,axis(p) freq_p;   u = x / sqrt(mean(x^2) + eps) w
//   a' = a cos - b sin, b' = b cos + a sin   for the pair (a, b) of u
//
// Everything between the loads and the one rounding to bf16 is 64 bits: a key
// goes on into 4 bits, where a last place of fp32 next to a rounding border
// would move a code by a whole step, and vector fp64 runs here at the rate of
// fp32.  So codes are those of the exactly rotated key, whatever order a
// kernel sums in.
//
// A head is D / 16 lanes of 16 channels: two pieces of 8 (16 bytes each, a
// head's pieces next to each other in a wave's load), chosen so that both
// channels of a pair lie in one lane.  A lane keeps its token's 8 cosines and
// sines and takes one head after the other.
#include "kv4_codes.h"

#include <cmath>

namespace svdq {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t rp_pack2(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// cos and sin of a (radians), in fp32 accuracy and better: a - q pi / 2 with
// the constant in two parts, then the Taylor series on [-pi / 4, pi / 4] (the
// terms left out are below 5e-17).
__device__ __forceinline__ void rp_cos_sin(double a, float &c, float &s)
{
    constexpr double kHi = 1.5707963267948966, kLo = 6.123233995736766e-17, kInv = 0.6366197723675814;
    const double q = __builtin_rint(a * kInv);
    const double r = __builtin_fma(-q, kLo, __builtin_fma(-q, kHi, a));
    const int n = (int)(q - 4.0 * __builtin_floor(q * 0.25));
    const double z = r * r;
    double ps = -1.0 / 1307674368000.0, pc = 1.0 / 20922789888000.0;
    ps = __builtin_fma(ps, z, 1.0 / 6227020800.0);
    ps = __builtin_fma(ps, z, -1.0 / 39916800.0);
    ps = __builtin_fma(ps, z, 1.0 / 362880.0);
    ps = __builtin_fma(ps, z, -1.0 / 5040.0);
    ps = __builtin_fma(ps, z, 1.0 / 120.0);
    ps = __builtin_fma(ps, z, -1.0 / 6.0);
    pc = __builtin_fma(pc, z, -1.0 / 87178291200.0);
    pc = __builtin_fma(pc, z, 1.0 / 479001600.0);
    pc = __builtin_fma(pc, z, -1.0 / 3628800.0);
    pc = __builtin_fma(pc, z, 1.0 / 40320.0);
    pc = __builtin_fma(pc, z, -1.0 / 720.0);
    pc = __builtin_fma(pc, z, 1.0 / 24.0);
    pc = __builtin_fma(pc, z, -0.5);
    const double sn = __builtin_fma(ps * z, r, r), cs = __builtin_fma(pc, z, 1.0);
    const float x = (float)(n & 1 ? sn : cs), y = (float)(n & 1 ? cs : sn);
    c = n == 1 || n == 2 ? -x : x;
    s = n & 2 ? -y : y;
}

// Four pairs of a token per thread.
__global__ __launch_bounds__(256) void rope_table_kernel(const int32_t *__restrict__ pos, int64_t n4, int axes,
                                                         const double *__restrict__ freq,
                                                         const int32_t *__restrict__ axis, int pairs,
                                                         float *__restrict__ cos, float *__restrict__ sin)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    const int q4 = pairs >> 2;
    const int64_t t = i / q4;
    const int p = 4 * (int)(i % q4);
    float c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int a = axis[p + k];
        const bool in = (uint32_t)a < (uint32_t)axes;
        const int at = pos[t * axes + (in ? a : 0)];
        rp_cos_sin(in ? (double)at * freq[p + k] : 0.0, c[k], s[k]);
    }
    reinterpret_cast<float4 *>(cos)[i] = make_float4(c[0], c[1], c[2], c[3]);
    reinterpret_cast<float4 *>(sin)[i] = make_float4(s[0], s[1], s[2], s[3]);
}

// Channels of a lane's two pieces, and the pairs that they hold.
template <int D, bool HALVES>
struct RopeLane {
    int a, b;            // first channels
    int pa, pb;          // first pairs of the cosines 0 .. 3 and 4 .. 7; >= pairs: not rotated
};

template <int D, bool HALVES>
__device__ __forceinline__ RopeLane<D, HALVES> rp_lane(int i, int pairs)
{
    RopeLane<D, HALVES> l;
    if (HALVES) {
        // pair p is (p, pairs + p); what lies behind 2 pairs is passed on
        const bool in = 8 * i < pairs;
        l.a = in ? 8 * i : 16 * i;
        l.b = in ? pairs + 8 * i : l.a + 8;
        l.pa = 8 * i, l.pb = 8 * i + 4;
    } else {
        l.a = 8 * i, l.b = D / 2 + 8 * i;
        l.pa = 4 * i, l.pb = D / 4 + 4 * i;
    }
    return l;
}

// A lane's eight cosines and sines of a token.
struct RopeTurn {
    double c[8], s[8];
};

template <int D, bool HALVES>
__device__ __forceinline__ RopeTurn rp_turn(const RopeArgs &r, const RopeLane<D, HALVES> &l, int t)
{
    const int row = r.index ? r.index[t] : t;
    const bool in = (uint32_t)row < (uint32_t)r.table_rows;
    RopeTurn o;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int p = h ? l.pb : l.pa;
        float4 c = make_float4(1.0f, 1.0f, 1.0f, 1.0f), s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in && p < r.pairs) {
            c = *reinterpret_cast<const float4 *>(r.cos + (int64_t)row * r.pairs + p);
            s = *reinterpret_cast<const float4 *>(r.sin + (int64_t)row * r.pairs + p);
        }
        o.c[4 * h] = c.x, o.c[4 * h + 1] = c.y, o.c[4 * h + 2] = c.z, o.c[4 * h + 3] = c.w;
        o.s[4 * h] = s.x, o.s[4 * h + 1] = s.y, o.s[4 * h + 2] = s.z, o.s[4 * h + 3] = s.w;
    }
    return o;
}

__device__ __forceinline__ void rp_unpack8(const uint4 &u, double *f)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bits_f32(w[i] << 16), f[2 * i + 1] = bits_f32(w[i] & 0xFFFF0000u);
}

// 1 / sqrt(x): the instruction's estimate and two Newton steps.
__device__ __forceinline__ double rp_rsqrt(double x)
{
    const double h = 0.5 * x;
    double y = __builtin_amdgcn_rsq(x);
    y *= __builtin_fma(-h * y, y, 1.5);
    return y * __builtin_fma(-h * y, y, 1.5);
}

// Norm (w given) and rotation of a lane's pieces xa, xb in place.
template <int D, bool HALVES>
__device__ __forceinline__ void rp_apply(uint4 &xa, uint4 &xb, const uint16_t *w, const RopeLane<D, HALVES> &l,
                                         const RopeTurn &r, double eps)
{
    double u[16];
    rp_unpack8(xa, u), rp_unpack8(xb, u + 8);
    double ss = 0.0;
#pragma unroll
    for (int k = 0; k < 16; ++k) ss = __builtin_fma(u[k], u[k], ss);
#pragma unroll
    for (int d = 1; d < D / 16; d <<= 1) ss += __shfl_xor(ss, d);
    if (w) {
        const double rs = rp_rsqrt(__builtin_fma(ss, 1.0 / D, eps));
        double g[16];
        rp_unpack8(*reinterpret_cast<const uint4 *>(w + l.a), g);
        rp_unpack8(*reinterpret_cast<const uint4 *>(w + l.b), g + 8);
#pragma unroll
        for (int k = 0; k < 16; ++k) u[k] = u[k] * rs * g[k];
    }
    float o[16];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int a = HALVES ? p : 2 * p, b = HALVES ? p + 8 : 2 * p + 1;
        o[a] = (float)__builtin_fma(u[a], r.c[p], -(u[b] * r.s[p]));
        o[b] = (float)__builtin_fma(u[b], r.c[p], u[a] * r.s[p]);
    }
    xa = make_uint4(rp_pack2(o[0], o[1]), rp_pack2(o[2], o[3]), rp_pack2(o[4], o[5]), rp_pack2(o[6], o[7]));
    xb = make_uint4(rp_pack2(o[8], o[9]), rp_pack2(o[10], o[11]), rp_pack2(o[12], o[13]), rp_pack2(o[14], o[15]));
}

// A wave's share of one token's heads: every parts-th set of 64 / (D / 16)
// heads, queries first, then keys (none of them in the cache's form).
template <int D, bool HALVES>
__device__ __forceinline__ void rp_rows(const RopeArgs &r, int64_t item, int lane)
{
    constexpr int L = D / 16, S = 64 / L;
    if (item >= (int64_t)r.T * r.parts) return;
    const int t = (int)(item / r.parts), part = (int)(item % r.parts);
    const RopeLane<D, HALVES> l = rp_lane<D, HALVES>(lane % L, r.pairs);
    const int heads = r.heads_q + r.heads_k, step = r.parts * S;
    int h = part * S + lane / L;
    auto source = [&](int hh) {
        const int g = min(hh, heads - 1);                  // heads past the last repeat it, never stored
        return g < r.heads_q ? r.Q + t * r.ldq + (int64_t)g * D : r.K + t * r.ldk + (int64_t)(g - r.heads_q) * D;
    };
    const uint16_t *p = source(h);
    uint4 na = *reinterpret_cast<const uint4 *>(p + l.a), nb = *reinterpret_cast<const uint4 *>(p + l.b);
    const RopeTurn turn = rp_turn(r, l, t);
    for (int h0 = part * S; h0 < heads; h0 += step, h += step) {
        uint4 xa = na, xb = nb;
        p = source(h + step);
        na = *reinterpret_cast<const uint4 *>(p + l.a), nb = *reinterpret_cast<const uint4 *>(p + l.b);
        rp_apply(xa, xb, h < r.heads_q ? r.wq : r.wk, l, turn, r.eps);
        if (h >= heads) continue;
        uint16_t *o = h < r.heads_q ? r.Qo + t * r.ldqo + (int64_t)h * D
                                    : r.Ko + t * r.ldko + (int64_t)(h - r.heads_q) * D;
        *reinterpret_cast<uint4 *>(o + l.a) = xa;
        *reinterpret_cast<uint4 *>(o + l.b) = xb;
    }
}

template <int D, bool HALVES>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(RopeArgs r)
{
    rp_rows<D, HALVES>(r, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), threadIdx.x & 63);
}

// The first kv_blocks blocks take a head of 2048 / D tokens' keys and values
// each: half of the threads norm and rotate the keys into LDS, then the tile
// goes the way of svdq_kv4_append.  The others take the queries.
template <bool INT4, int D, bool HALVES>
__global__ __launch_bounds__(KC_THREADS) void kv4_rope_append_kernel(Kv4View c, RopeArgs r,
                                                                     const uint16_t *__restrict__ V, int64_t ldv,
                                                                     const int32_t *__restrict__ slots,
                                                                     uint32_t kv_blocks)
{
    constexpr int TPT = D / 8, TB = KcTile<D>::TB, L = D / 16, ROW = D + 8;
    __shared__ KcTile<D> m;
    __shared__ __attribute__((aligned(16))) uint16_t kr[TB * ROW];
    const int tid = threadIdx.x;
    if (blockIdx.x >= kv_blocks) {
        rp_rows<D, HALVES>(r, (int64_t)(blockIdx.x - kv_blocks) * 4 + (tid >> 6), tid & 63);
        return;
    }
    const int head = blockIdx.x % c.heads, t0 = (int)(blockIdx.x / c.heads) * TB;
    const int tk = tid / TPT, q = tid % TPT;
    if (tid < TB) m.sl[tid] = t0 + tid < r.T ? slots[t0 + tid] : -1;
    const uint4 vv = *reinterpret_cast<const uint4 *>(V + min(t0 + tk, r.T - 1) * ldv + (int64_t)head * D + 8 * q);
    if (tid < TB * L) {
        const int t = min(t0 + tid / L, r.T - 1);
        const RopeLane<D, HALVES> l = rp_lane<D, HALVES>(tid % L, r.pairs);
        const uint16_t *p = r.K + t * r.ldk + (int64_t)head * D;
        uint4 xa = *reinterpret_cast<const uint4 *>(p + l.a), xb = *reinterpret_cast<const uint4 *>(p + l.b);
        rp_apply(xa, xb, r.wk, l, rp_turn(r, l, t), r.eps);
        *reinterpret_cast<uint4 *>(kr + tid / L * ROW + l.a) = xa;
        *reinterpret_cast<uint4 *>(kr + tid / L * ROW + l.b) = xb;
    }
    float fk[8], fv[8];
    kc_unpack8(vv, fv);
    __syncthreads();
    kc_unpack8(*reinterpret_cast<const uint4 *>(kr + tk * ROW + 8 * q), fk);
    kc_store_tile<INT4, D>(c, head, m, fk, fv, tid);
}

// Waves per token: as many as give eight waves per compute unit, at most one
// per set of heads.
int rope_parts(int T, int heads, int D)
{
    const int sets = (heads + 64 / (D / 16) - 1) / (64 / (D / 16));
    const int64_t want = (8 * (int64_t)device_cu_count() + T - 1) / T;
    return (int)(want < sets ? want : sets);
}

}  // namespace

void rope_frequencies(const int *sections, int axes, double theta, svdq_rope_axes layout, double *freq, int32_t *axis)
{
    int pairs = 0;
    for (int a = 0; a < axes; ++a) pairs += sections[a];
    int p = 0;
    for (int a = 0; a < axes; ++a)
        for (int j = 0; j < sections[a]; ++j, ++p) {
            axis[p] = a;
            freq[p] = layout == SVDQ_ROPE_AXES_BLOCKS ? std::pow(theta, -(double)j / sections[a])
                                                      : std::pow(theta, -(double)p / pairs);
        }
    if (layout == SVDQ_ROPE_AXES_INTERLEAVED)
        for (p = 0; p < pairs; ++p) axis[p] = p / axes < sections[p % axes] ? p % axes : 0;
}

hipError_t launch_rope_table(const int32_t *pos, int T, int axes, const double *freq, const int32_t *axis, int pairs,
                             float *cos, float *sin, hipStream_t stream)
{
    const int64_t n4 = (int64_t)T * (pairs / 4);
    rope_table_kernel<<<(uint32_t)((n4 + 255) / 256), 256, 0, stream>>>(pos, n4, axes, freq, axis, pairs, cos, sin);
    return hipGetLastError();
}

hipError_t launch_qk_norm_rope(RopeArgs r, int dim, bool halves, hipStream_t stream)
{
    r.parts = rope_parts(r.T, r.heads_q + r.heads_k, dim);
    const uint32_t grid = (uint32_t)(((int64_t)r.T * r.parts + 3) / 4);
    if (dim == 64) halves ? qk_norm_rope_kernel<64, true><<<grid, 256, 0, stream>>>(r) : qk_norm_rope_kernel<64, false><<<grid, 256, 0, stream>>>(r);
    else if (dim == 128) halves ? qk_norm_rope_kernel<128, true><<<grid, 256, 0, stream>>>(r) : qk_norm_rope_kernel<128, false><<<grid, 256, 0, stream>>>(r);
    else halves ? qk_norm_rope_kernel<256, true><<<grid, 256, 0, stream>>>(r) : qk_norm_rope_kernel<256, false><<<grid, 256, 0, stream>>>(r);
    return hipGetLastError();
}

hipError_t launch_kv4_rope_append(const Kv4View &c, RopeArgs r, bool halves, const uint16_t *V, int64_t ldv,
                                  const int32_t *slots, hipStream_t stream)
{
    r.heads_k = 0;                                         // the waves of rows take the queries alone
    r.parts = rope_parts(r.T, r.heads_q, c.dim);
    const int tb = 2048 / c.dim;
    const uint32_t kv = (uint32_t)((r.T + tb - 1) / tb) * c.heads;
    const uint32_t grid = kv + (uint32_t)(((int64_t)r.T * r.parts + 3) / 4);
#define RP_LAUNCH(I, D) \
    (halves ? kv4_rope_append_kernel<I, D, true><<<grid, KC_THREADS, 0, stream>>>(c, r, V, ldv, slots, kv) \
            : kv4_rope_append_kernel<I, D, false><<<grid, KC_THREADS, 0, stream>>>(c, r, V, ldv, slots, kv))
    if (c.int4 && c.dim == 64) RP_LAUNCH(true, 64);
    else if (c.int4) RP_LAUNCH(true, 128);
    else if (c.dim == 64) RP_LAUNCH(false, 64);
    else RP_LAUNCH(false, 128);
#undef RP_LAUNCH
    return hipGetLastError();
}

}  // namespace svdq
