// rope.hip -- rotary positions with several axes: their tables, and the norm
// and rotation of query and key heads, on their own or on the way into the
// 4-bit cache.
//
//   angle_tp = pos_t,axis(p) freq_p;   u = x / sqrt(mean(x^2) + eps) w
//   a' = a cos - b sin, b' = b cos + a sin   for the pair (a, b) of u
//
// Keys: everything between the loads and the one rounding to bf16 is 64 bits.  A
// key goes on into 4 bits, where a last place of fp32 next to a rounding border
// would move a code by a whole step; so its codes are those of the exactly rotated
// key, whatever order a kernel sums in, and the two kernels agree.  Queries end in
// bf16 and are fp32 (the conversions to and from fp64 took most of the time), but
// for heads whose squares leave its range.
//
// A head is D / 16 lanes of 16 channels: two pieces of 8 (16 bytes each, a
// head's pieces next to each other in a wave's load), chosen so that both
// channels of a pair lie in one lane.  A lane keeps its token's 8 cosines and
// sines and takes one head after the other.
//
// What bounds it, and what it measured: 4608 tokens, 48 heads of 128, norm: 23.2
// us for 116 MB = 5.0 TB/s, a large copy's rate (5.1), the same heads again and again
// 20.9 (of 48 pairs 20.6); keys and queries alike in 64 bits 25.6 (conversions).  The
// table of their angles 3.2 us.  4063 tokens, 28 + 4 heads of queries and keys, 4 of
// values, into the INT4 cache: 17.8 us for 71 MB: the keys' and values' blocks (64
// bits, then the quantizer) beside the copy.  One token, 32 heads over 8: 4.1 us, a
// launch and loads in turn.
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

__global__ __launch_bounds__(256) void rope_table_kernel(const int32_t *__restrict__ pos, int64_t n, int axes,
                                                         const double *__restrict__ freq,
                                                         const int32_t *__restrict__ axis, int pairs,
                                                         float *__restrict__ cos, float *__restrict__ sin)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t t = i / pairs;
    const int p = (int)(i % pairs), a = axis[p];
    const bool in = (uint32_t)a < (uint32_t)axes;
    const int at = pos[t * axes + (in ? a : 0)];
    rp_cos_sin(in ? (double)at * freq[p] : 0.0, cos[i], sin[i]);
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

// A lane's eight cosines and sines of a token, those of four pairs each turned or
// not; some: a lane of the wave has pairs that are not.
struct RopeTurn {
    float c[8], s[8];
    bool on[2], some;
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
        o.on[h] = in && p < r.pairs;
        if (o.on[h]) {
            c = *reinterpret_cast<const float4 *>(r.cos + (int64_t)row * r.pairs + p);
            s = *reinterpret_cast<const float4 *>(r.sin + (int64_t)row * r.pairs + p);
        }
        o.c[4 * h] = c.x, o.c[4 * h + 1] = c.y, o.c[4 * h + 2] = c.z, o.c[4 * h + 3] = c.w;
        o.s[4 * h] = s.x, o.s[4 * h + 1] = s.y, o.s[4 * h + 2] = s.z, o.s[4 * h + 3] = s.w;
    }
    o.some = __any(!o.on[0] || !o.on[1]);
    return o;
}

template <class F>
__device__ __forceinline__ void rp_unpack8(const uint4 &u, F *f)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bits_f32(w[i] << 16), f[2 * i + 1] = bits_f32(w[i] & 0xFFFF0000u);
}

// 1 / sqrt(x): fp64 from the instruction's estimate by two Newton steps (which
// would make 0 inf of the zero that an infinity has).
__device__ __forceinline__ double rp_rsqrt(double x)
{
    const double h = 0.5 * x, e = __builtin_amdgcn_rsq(x);
    double y = e * __builtin_fma(-h * e, e, 1.5);
    y *= __builtin_fma(-h * y, y, 1.5);
    return e == 0.0 ? 0.0 : y;
}
__device__ __forceinline__ float rp_rsqrt(float x) { return __builtin_amdgcn_rsqf(x); }

__device__ __forceinline__ double rp_fma(double a, double b, double c) { return __builtin_fma(a, b, c); }
__device__ __forceinline__ float rp_fma(float a, float b, float c) { return __builtin_fmaf(a, b, c); }

// Norm (with the lane's weights g, if there is one) and rotation of a lane's pieces
// xa, xb, into ya, yb.  fp32: true where the head has a sum of squares that fp32 may
// not hold to its last places.
template <class F, int D, bool HALVES>
__device__ __forceinline__ bool rp_apply(const uint4 &xa, const uint4 &xb, uint4 &ya, uint4 &yb, bool norm,
                                         const uint4 &ga, const uint4 &gb, const RopeTurn &r, double eps)
{
    F u[16];
    bool out = false;
    rp_unpack8(xa, u), rp_unpack8(xb, u + 8);
    if (norm) {
        F ss = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) ss = rp_fma(u[k], u[k], ss);
#pragma unroll
        for (int d = 1; d < D / 16; d <<= 1) ss += __shfl_xor(ss, d);
        out = sizeof(F) == 4 && !(ss > (F)1e-25 && ss < (F)1e35);
        const F rs = rp_rsqrt(rp_fma(ss, (F)(1.0 / D), (F)eps));
        F g[16];
        rp_unpack8(ga, g), rp_unpack8(gb, g + 8);
#pragma unroll
        for (int k = 0; k < 16; ++k) u[k] = u[k] * rs * g[k];
    }
    float o[16];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int a = HALVES ? p : 2 * p, b = HALVES ? p + 8 : 2 * p + 1;
        const F c = r.c[p], s = r.s[p];
        o[a] = (float)rp_fma(u[a], c, -(u[b] * s));
        o[b] = (float)rp_fma(u[b], c, u[a] * s);
    }
    if (r.some) {                                          // not by 1 and 0: an infinity would reach its neighbour
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const bool on = r.on[HALVES ? (k & 7) >> 2 : k >> 3];
            o[k] = on ? o[k] : (float)u[k];
        }
    }
    ya = make_uint4(rp_pack2(o[0], o[1]), rp_pack2(o[2], o[3]), rp_pack2(o[4], o[5]), rp_pack2(o[6], o[7]));
    yb = make_uint4(rp_pack2(o[8], o[9]), rp_pack2(o[10], o[11]), rp_pack2(o[12], o[13]), rp_pack2(o[14], o[15]));
    return out;
}

// A lane's norm weights.
template <int D, bool HALVES>
__device__ __forceinline__ void rp_weights(const uint16_t *w, const RopeLane<D, HALVES> &l, uint4 &ga, uint4 &gb)
{
    ga = gb = make_uint4(0u, 0u, 0u, 0u);
    if (w) ga = *reinterpret_cast<const uint4 *>(w + l.a), gb = *reinterpret_cast<const uint4 *>(w + l.b);
}

// One token's heads of one kind, sets first, first + step, .. of 64 / (D / 16) heads
// each.
template <class F, int D, bool HALVES>
__device__ __forceinline__ void rp_heads(const uint16_t *x, uint16_t *y, int heads, int first, int step,
                                         const uint16_t *w, const RopeLane<D, HALVES> &l, const RopeTurn &turn,
                                         double eps, int lane)
{
    constexpr int L = D / 16, S = 64 / L;
    uint4 ga, gb;
    rp_weights<D, HALVES>(w, l, ga, gb);
    auto load = [&](int set, uint4 &a, uint4 &b) {
        const int64_t h = min(set * S + lane / L, heads - 1);      // heads past the last repeat it, never stored
        a = *reinterpret_cast<const uint4 *>(x + h * D + l.a), b = *reinterpret_cast<const uint4 *>(x + h * D + l.b);
    };
    uint4 na, nb;
    load(first, na, nb);
    for (int set = first; set * S < heads; set += step) {
        const uint4 xa = na, xb = nb;
        uint4 ya, yb;
        load(set + step, na, nb);
        const bool out = rp_apply<F, D, HALVES>(xa, xb, ya, yb, w != nullptr, ga, gb, turn, eps);
        if (__any(out)) {                                  // for these heads alone: the others' bits stay
            uint4 za, zb;
            rp_apply<double, D, HALVES>(xa, xb, za, zb, true, ga, gb, turn, eps);
            if (out) ya = za, yb = zb;
        }
        const int64_t h = set * S + lane / L;
        if (h >= heads) continue;
        *reinterpret_cast<uint4 *>(y + h * D + l.a) = ya;
        *reinterpret_cast<uint4 *>(y + h * D + l.b) = yb;
    }
}

// A wave's share of one token: every parts-th set of heads, queries, then keys.
template <int D, bool HALVES>
__device__ __forceinline__ void rp_rows(const RopeArgs &r, int64_t item, int lane)
{
    constexpr int L = D / 16, S = 64 / L;
    if (item >= (int64_t)r.T * r.parts) return;
    const int t = (int)(item / r.parts), part = (int)(item % r.parts);
    const RopeLane<D, HALVES> l = rp_lane<D, HALVES>(lane % L, r.pairs);
    const RopeTurn turn = rp_turn(r, l, t);
    const int nq = (r.heads_q + S - 1) / S;
    if (part < nq)
        rp_heads<float, D, HALVES>(r.Q + t * r.ldq, r.Qo + t * r.ldqo, r.heads_q, part, r.parts, r.wq, l, turn, r.eps, lane);
    // the keys' sets follow the queries'
    const int first = part >= nq ? part - nq : (r.parts - (nq - part) % r.parts) % r.parts;
    if (r.heads_k > 0 && first * S < r.heads_k)
        rp_heads<double, D, HALVES>(r.K + t * r.ldk, r.Ko + t * r.ldko, r.heads_k, first, r.parts, r.wk, l, turn, r.eps, lane);
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
        const uint4 xa = *reinterpret_cast<const uint4 *>(p + l.a), xb = *reinterpret_cast<const uint4 *>(p + l.b);
        uint4 ga, gb, ya, yb;
        rp_weights<D, HALVES>(r.wk, l, ga, gb);
        rp_apply<double, D, HALVES>(xa, xb, ya, yb, r.wk != nullptr, ga, gb, rp_turn(r, l, t), r.eps);
        *reinterpret_cast<uint4 *>(kr + tid / L * ROW + l.a) = ya;
        *reinterpret_cast<uint4 *>(kr + tid / L * ROW + l.b) = yb;
    }
    float fk[8], fv[8];
    kc_unpack8(vv, fv);
    __syncthreads();
    kc_unpack8(*reinterpret_cast<const uint4 *>(kr + tk * ROW + 8 * q), fk);
    kc_store_tile<INT4, D>(c, head, m, fk, fv, tid);
}

// Waves per token: as many as give eight waves per compute unit, at most one
// per set of heads.
int rope_parts(int T, int heads_q, int heads_k, int D)
{
    const int S = 64 / (D / 16), sets = (heads_q + S - 1) / S + (heads_k + S - 1) / S;
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
    const int64_t n = (int64_t)T * pairs;
    rope_table_kernel<<<(uint32_t)((n + 255) / 256), 256, 0, stream>>>(pos, n, axes, freq, axis, pairs, cos, sin);
    return hipGetLastError();
}

hipError_t launch_qk_norm_rope(RopeArgs r, int dim, bool halves, hipStream_t stream)
{
    r.parts = rope_parts(r.T, r.heads_q, r.heads_k, dim);
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
    r.parts = rope_parts(r.T, r.heads_q, 0, c.dim);
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
