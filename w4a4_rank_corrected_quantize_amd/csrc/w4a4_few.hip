// w4a4_few.hip -- the W4A4 linear for few rows (up to 64): decoding steps and
// trees of drafted tokens, where the product is one pass over the weights.
//
//   y_mn = sum_g sx_mg sw_ng P_mng + sum_j h_mj up[n][j] + b_n   [GELU-tanh]
//   gated: y_mf = act(gate_mf) up_mf, the two rows f and F + f of the weight
//
// A block owns 16 RT output rows of the weight (gated: 8 RT channels, their
// gate and up rows) and all rows of X; its waves take the row's 128-byte lines
// in turn.  A wave's stage is one line (256 channels) of 16 RT weight rows and
// 16 CT rows of X with their scales.  It reaches LDS by DMA in whole lines (8
// lanes per line), DEPTH stages ahead, in a ring of the wave's own: no barrier
// until the waves' fp32 sums meet.
//
// Products.  MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4 takes codes and E8M0
// scales as they are.  INT4: a group's 64 codes, widened to exact E4M3 bytes (q
// 2^-9), are two v_mfma_f32_16x16x32_fp8_fp8, whose sum is the exact group dot
// product 2^-18; one fp32 product of the two scales and one fma per group.  The
// order of k inside a group is a permutation that both operands share.
//
// The waves' sums are added in wave order; the low-rank term (h in bf16 high and
// low parts) and the epilogue follow in fp32, rounded once.  Results depend on
// the sizes alone.
#include "svdq_internal.h"
#include "svdq_quant.h"
#include "w4a4_epilogue.h"

namespace svdq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) uint8_t fw_lds_u8;

__device__ __forceinline__ uint32_t fw_lds(const void *p)
{
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const fw_lds_u8 *)p);
}

// One LDS-DMA load per lane: 16 bytes, 4 bytes, or one byte (as a dword), from
// base + off to lds + 16 (4, 4) * lane.  M0 is saved and restored around it.
#define FW_DMA(NAME, OP)                                                                                             \
    __device__ __forceinline__ void NAME(uint32_t lds, uint32_t off, const void *base)                                \
    {                                                                                                                \
        uint32_t keep;                                                                                               \
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t" OP " %2, %3\n\ts_mov_b32 m0, %0"           \
                     : "=&s"(keep) : "s"(lds), "v"(off), "s"(base) : "memory");                                       \
    }
FW_DMA(fw_dma16, "global_load_lds_dwordx4")
FW_DMA(fw_dma4, "global_load_lds_dword")
FW_DMA(fw_dma1, "global_load_lds_ubyte")
#undef FW_DMA

struct FewArgs {
    const uint8_t *xq, *wq;
    const void *xscale, *wscale;
    const float *h;
    const uint16_t *up, *bias;
    uint16_t *Y;
    int M, N, K, act;                   // act: FEW_*
};
constexpr int FEW_NONE = 0, FEW_GELU = 1, FEW_SILU = 2;

// Bytes of a tile of 16 rows in a stage: a line of codes per row, then its
// scales (INT4: fp32 [4 groups][16 rows]; MXFP4: a dword per lane and product).
template <bool INT4>
struct FewTile {
    static constexpr int kCodes = 16 * 128, kScales = INT4 ? 256 : 512, kBytes = kCodes + kScales;
    static constexpr int kLoads = INT4 ? 3 : 4;
};

// 16-byte segment s of row r lies at s ^ (r / 2 % 8): 16 rows' reads of a
// segment fall into 16 different bank groups of the LDS (64 banks).
__device__ __forceinline__ int fw_seg(int r, int s) { return s ^ ((r >> 1) & 7); }

// Issues the loads of a tile's stage: `row` is the lane's row of the matrix for
// its two lines' lanes (code[j]) and its scales (srow).  Past the end of a row
// the last segment is read again.
struct FewRows {
    uint32_t code[2], scale;            // byte offsets of the lane's rows
};

template <bool INT4>
__device__ __forceinline__ void fw_issue(uint32_t lds, const FewRows &o, const uint8_t *q, const void *scales, int st,
                                         int segs, int lane)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = 8 * j + (lane >> 3);
        const int s = min(8 * st + fw_seg(r, lane & 7), segs - 1);
        fw_dma16(lds + 1024 * j, o.code[j] + 16 * s, q);
    }
    lds += FewTile<INT4>::kCodes;
    if constexpr (INT4) {
        fw_dma4(lds, o.scale + 4 * min(4 * st + (lane >> 4), segs / 2 - 1), scales);
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) fw_dma1(lds + 256 * s, o.scale + min(8 * st + 2 * (lane >> 4) + s, segs - 1), scales);
    }
}

template <int N>
__device__ __forceinline__ void fw_wait()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// 8 code bytes -> 16 E4M3 bytes: operands of two products.
__device__ __forceinline__ void fw_widen(uint2 w, long &a, long &b)
{
    const uint32_t e0 = (w.x & 0x07070707u) | ((w.x & 0x08080808u) << 4), o0 = ((w.x >> 4) & 0x07070707u) | (w.x & 0x80808080u);
    const uint32_t e1 = (w.y & 0x07070707u) | ((w.y & 0x08080808u) << 4), o1 = ((w.y >> 4) & 0x07070707u) | (w.y & 0x80808080u);
    a = (long)((uint64_t)o0 << 32 | e0);
    b = (long)((uint64_t)o1 << 32 | e1);
}

template <bool INT4, int RT, int CT, bool GATED, int W, int DEPTH>
__global__ __launch_bounds__(64 * W) void w4a4_few_kernel(FewArgs a)
{
    typedef FewTile<INT4> Tile;
    constexpr int STAGE = (RT + CT) * Tile::kBytes, NL = (RT + CT) * Tile::kLoads;
    constexpr int RING = W * DEPTH * STAGE, SUMS = W * RT * CT * 1024;
    static_assert(NL * (DEPTH - 1) <= 63, "the loads in flight are counted in 6 bits");
    __shared__ __attribute__((aligned(16))) uint8_t lds[RING > SUMS ? RING : SUMS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j16 = lane & 15, b = lane >> 4;
    constexpr int NT = GATED ? RT / 2 : RT;              // tiles of output channels
    const int n0 = blockIdx.x * (16 * NT);
    const int KB = a.K >> 1, segs = KB >> 4, stages = (segs + 7) >> 3;
    const int srow = INT4 ? 4 * (a.K >> 6) : a.K >> 5;   // bytes of a row's scales

    // row of the weight: tile t, row r
    auto wrow = [&](int t, int r) {
        const int n = min(n0 + 16 * (GATED ? t >> 1 : t) + r, a.N - 1);
        return GATED && (t & 1) ? a.N + n : n;
    };
    FewRows wo[RT], xo[CT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) wo[t].code[j] = (uint32_t)wrow(t, 8 * j + (lane >> 3)) * KB;
        wo[t].scale = (uint32_t)wrow(t, j16) * srow;
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
#pragma unroll
        for (int j = 0; j < 2; ++j) xo[c].code[j] = (uint32_t)min(16 * c + 8 * j + (lane >> 3), a.M - 1) * KB;
        xo[c].scale = (uint32_t)min(16 * c + j16, a.M - 1) * srow;
    }
    uint8_t *ring = lds + wave * (DEPTH * STAGE);
    const uint32_t ring0 = fw_lds(ring);
    auto issue = [&](int i) {
        const int st = wave + i * W;
        const uint32_t at = ring0 + (uint32_t)(i % DEPTH) * STAGE;
#pragma unroll
        for (int t = 0; t < RT; ++t) fw_issue<INT4>(at + t * Tile::kBytes, wo[t], a.wq, a.wscale, st, segs, lane);
#pragma unroll
        for (int c = 0; c < CT; ++c) fw_issue<INT4>(at + (RT + c) * Tile::kBytes, xo[c], a.xq, a.xscale, st, segs, lane);
    };
    const int mine = wave < stages ? (stages - wave + W - 1) / W : 0;

    f32x4 acc[RT][CT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
        if (i < mine) issue(i);
    for (int i = 0; i < mine; ++i) {
        // this stage's loads are done: all but those of the stages after it
        const int after = min(DEPTH - 1, mine - 1 - i);
        if (after == 0) fw_wait<0>();
        else if (after == 1) fw_wait<NL>();
        else if (DEPTH > 3 && after == 3) fw_wait<NL * (DEPTH > 3 ? 3 : 0)>();
        else if (DEPTH > 2) fw_wait<NL * (DEPTH > 2 ? 2 : 0)>();
        const uint8_t *S = ring + (i % DEPTH) * STAGE;
        const int st = wave + i * W;
        if constexpr (INT4) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (4 * st + g >= (segs >> 1)) break;
                const int at = j16 * 128 + 16 * fw_seg(j16, 2 * g + (b >> 1)) + 8 * (b & 1);
                long x0[CT], x1[CT];
                float sx[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const uint8_t *p = S + (RT + c) * Tile::kBytes;
                    fw_widen(*reinterpret_cast<const uint2 *>(p + at), x0[c], x1[c]);
                    sx[c] = *reinterpret_cast<const float *>(p + Tile::kCodes + 4 * (16 * g + j16));
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint8_t *p = S + t * Tile::kBytes;
                    long w0, w1;
                    fw_widen(*reinterpret_cast<const uint2 *>(p + at), w0, w1);
                    const f32x4 sw = *reinterpret_cast<const f32x4 *>(p + Tile::kCodes + 4 * (16 * g + 4 * b));
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
                        d = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(w0, x0[c], d, 0, 0, 0);
                        d = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(w1, x1[c], d, 0, 0, 0);
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[t][c][k] = __builtin_fmaf(d[k], sw[k] * sx[c], acc[t][c][k]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int at = j16 * 128 + 16 * fw_seg(j16, 2 * b + s);
                const bool in = 8 * st + 2 * b + s < segs;      // segments past the row's end: zeros of X
                i32x8 x[CT];
                int ex[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const uint8_t *p = S + (RT + c) * Tile::kBytes;
                    const uint4 v = *reinterpret_cast<const uint4 *>(p + at);
                    x[c] = (i32x8){in ? (int)v.x : 0, in ? (int)v.y : 0, in ? (int)v.z : 0, in ? (int)v.w : 0, 0, 0, 0, 0};
                    ex[c] = *reinterpret_cast<const int *>(p + Tile::kCodes + 256 * s + 4 * lane);
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint8_t *p = S + t * Tile::kBytes;
                    const uint4 v = *reinterpret_cast<const uint4 *>(p + at);
                    const i32x8 w = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
                    const int ew = *reinterpret_cast<const int *>(p + Tile::kCodes + 256 * s + 4 * lane);
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        acc[t][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x[c], acc[t][c], 4, 4, 0, ew, 0, ex[c]);
                }
            }
        }
        if (i + DEPTH < mine) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage has been read: its place is free
            issue(i + DEPTH);
        }
    }
    // the waves' sums: tile (t, c) of wave w at w RT CT + t CT + c
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) sums[64 * ((wave * RT + t) * CT + c) + lane] = acc[t][c];
    __syncthreads();
    // wave u finishes the output tiles u, u + W, ..: lane (j16, b) has channels
    // 4 b .. 4 b + 3 of row j16
    for (int u = wave; u < NT * CT; u += W) {
        const int c = u % CT, m = 16 * c + j16, mc = min(m, a.M - 1);
        bf16x8 hhi, hlo;
        float hv[8];
        load_h8(a.h, mc, a.M, 8 * b, hv);
        split_h(hv, hhi, hlo);
        f32x4 y[GATED ? 2 : 1];
#pragma unroll
        for (int k = 0; k < (GATED ? 2 : 1); ++k) {
            const int t = GATED ? 2 * (u / CT) + k : u / CT;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < W; ++w) v += sums[64 * ((w * RT + t) * CT + c) + lane];
            if (INT4) v *= 262144.0f;
            const bf16x8 ua = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(a.up + (size_t)wrow(t, j16) * 32 + 8 * b));
            v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ua, hhi, v, 0, 0, 0);
            v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ua, hlo, v, 0, 0, 0);
            if (a.bias) {
                const uint2 bi = *reinterpret_cast<const uint2 *>(a.bias + min((int)(n0 + 16 * (GATED ? t >> 1 : t) + 4 * b), a.N - 4) + (GATED && k ? a.N : 0));
                v[0] += bf16_to_f32(bi.x & 0xFFFFu), v[1] += bf16_to_f32(bi.x >> 16);
                v[2] += bf16_to_f32(bi.y & 0xFFFFu), v[3] += bf16_to_f32(bi.y >> 16);
            }
            y[k] = v;
        }
        const int n = n0 + 16 * (u / CT) + 4 * b;
        if (m >= a.M || n >= a.N) continue;
        f32x4 o = y[0];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (a.act == FEW_GELU) o[k] = gelu_tanh(o[k]);
            else if (a.act == FEW_SILU) o[k] = silu(o[k]);
            if (GATED) o[k] *= y[GATED ? 1 : 0][k];
        }
        *reinterpret_cast<uint2 *>(a.Y + (size_t)m * a.N + n) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
}

template <bool INT4, int CT, bool GATED>
void few_launch(const FewArgs &a, hipStream_t stream)
{
    constexpr int RT = GATED ? 2 : 1, NT = GATED ? RT / 2 : RT;
    constexpr int W = CT == 4 ? 4 : 8, DEPTH = CT == 1 && !GATED ? 3 : 2;
    const uint32_t grid = (uint32_t)((a.N + 16 * NT - 1) / (16 * NT));
    w4a4_few_kernel<INT4, RT, CT, GATED, W, DEPTH><<<grid, 64 * W, 0, stream>>>(a);
}

template <bool INT4, bool GATED>
void few_rows(const FewArgs &a, hipStream_t stream)
{
    if (a.M <= 16) few_launch<INT4, 1, GATED>(a, stream);
    else if (a.M <= 32) few_launch<INT4, 2, GATED>(a, stream);
    else few_launch<INT4, 4, GATED>(a, stream);
}

}  // namespace

hipError_t launch_w4a4_few(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                           const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N, int K,
                           svdq_precision prec, svdq_epilogue epi, uint16_t *Y, hipStream_t stream)
{
    const FewArgs a{xq, wq, xscale, wscale, h, up, bias, Y, M, N, K, epi == SVDQ_EPI_GELU_TANH ? FEW_GELU : FEW_NONE};
    if (prec == SVDQ_INT4) few_rows<true, false>(a, stream);
    else few_rows<false, false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_w4a4_few_gated(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                                 const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N, int K,
                                 svdq_precision prec, svdq_activation act, uint16_t *Y, hipStream_t stream)
{
    const FewArgs a{xq, wq, xscale, wscale, h, up, bias, Y, M, N, K, act == SVDQ_ACT_GELU_TANH ? FEW_GELU : FEW_SILU};
    if (prec == SVDQ_INT4) few_rows<true, true>(a, stream);
    else few_rows<false, true>(a, stream);
    return hipGetLastError();
}

}  // namespace svdq
