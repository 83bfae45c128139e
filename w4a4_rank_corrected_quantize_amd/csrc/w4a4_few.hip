// w4a4_few.hip -- the W4A4 linear for few rows: decoding steps and trees of
// drafted tokens, where the product is one pass over the weights (one per 64
// rows).
//
//   y_mn = sum_g sx_mg sw_ng P_mng + sum_j h_mj up[n][j] + b_n   [GELU-tanh]
//   gated: y_mf = act(gate_mf) up_mf, the two rows f and F + f of the weight
//
// A block owns WN sets of 16 RT rows of the weight (gated: 8 RT channels, their
// gate and up rows) and up to 64 rows of X; WK waves per set take the rows'
// 128-byte lines in turn.  A wave's stage is one line (256 channels) of its set's
// rows and of 16 CT rows of X, with their scales.  It reaches LDS by DMA in whole
// lines (8 lanes per line), several stages ahead.  One row of X up to a few are
// kept whole in LDS instead; with one set per block the ring is the wave's own and
// needs no barrier until the waves' fp32 sums meet, with two they share the lines
// of X.
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
//
// What bounds it, and what it measured (in a graph; weights out of the HBM, over 1
// GB of others in between / three sets in turn, which the last-level cache holds in
// part):
//   1 x 4096 -> 2 x 14336, MXFP4: 14.9 / 11.7 us for 64 MB = 4.3 TB/s: the memory;
//   INT4 18.4 / 14.7 us for 68 MB, the widening of the codes beside it.
//   1 x 4096 -> 6144, INT4: 6.8 / 6.3 us for 14.6 MB: 384 blocks of one wave's length,
//   a launch (2.5 us), two latencies of memory and the sum of eight waves.
//   48 x 11008 -> 4096, MXFP4: 12.7 / 9.7 us for 24.9 MB: every block reads all of X
//   from the L2 (68 MB in all) next to its weights; INT4 16.1 / 13.3, 48 x 14336 20.2 /
//   16.3: every wave widens its lines of X for one tile of channels.
//   64 x 4096 -> 2 x 14336: MXFP4 21.9 / 17.5, INT4 40.1 / 36.1 us, the widening.
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
    int chunks;                         // sets of 16 CT rows, set by the launch
};
constexpr int FEW_NONE = 0, FEW_GELU = 1, FEW_SILU = 2;

// Forms: INT4; MXFP4 with rows of scales that start on 4 bytes (K % 128 == 0);
// MXFP4 with rows of scales that start anywhere.
constexpr int FEW_INT4 = 0, FEW_MX = 1, FEW_MX_ODD = 2;

// Bytes of a tile of 16 rows in a stage: a line of codes per row, then its scales:
// fp32 [4 groups][16 rows]; dwords of four blocks [2][16 rows]; a dword per block,
// lane and product.
template <int FORM>
struct FewTile {
    static constexpr int kCodes = 16 * 128, kScales = FORM == FEW_INT4 ? 256 : FORM == FEW_MX ? 128 : 512;
    static constexpr int kBytes = kCodes + kScales, kLoads = FORM == FEW_MX_ODD ? 4 : 3;
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

// PARTS waves share the loads of a tile: part p has the lines of rows 8 p .. and
// half of the scales.
template <int FORM, int PARTS = 1>
__device__ __forceinline__ void fw_issue(uint32_t lds, const FewRows &o, const uint8_t *q, const void *scales, int st,
                                         int segs, int lane, int part = 0)
{
    static_assert(PARTS == 1 || PARTS == 2, "a tile's two loads of lines");
    auto line = [&](int j) {
        const int s = min(8 * st + fw_seg(8 * j + (lane >> 3), lane & 7), segs - 1);
        fw_dma16(lds + 1024 * j, (j ? o.code[1] : o.code[0]) + 16 * s, q);
    };
    if (PARTS == 1 || part == 0) line(0);
    if (PARTS == 1 || part == 1) line(1);
    lds += FewTile<FORM>::kCodes;
    if constexpr (FORM == FEW_INT4) {
        if (PARTS == 1 || lane >> 5 == part) fw_dma4(lds, o.scale + 4 * min(4 * st + (lane >> 4), segs / 2 - 1), scales);
    } else if constexpr (FORM == FEW_MX) {
        if (PARTS == 1 ? lane < 32 : lane >> 4 == part) fw_dma4(lds, o.scale + 4 * min(2 * st + (lane >> 4), segs / 4 - 1), scales);
    } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (PARTS == 1 || part == s) fw_dma1(lds + 256 * s, o.scale + min(8 * st + 2 * (lane >> 4) + s, segs - 1), scales);
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

// X kept whole in LDS: row r at r * fw_xrow, its 16-byte unit u at u ^ (r % 16);
// then the rows' scales as dwords (INT4: fp32; MXFP4: a byte each), an odd number
// apart: 16 rows' reads fall into different banks.  INT4 with room for it: then
// the rows once more, widened, 16 bytes for every 8, in the same order (once per
// block instead of by every wave and tile).
__host__ __device__ constexpr int fw_xrow(int K) { return ((K >> 1) + 255) & ~255; }
__host__ __device__ constexpr int fw_xwide(int K) { return (K + 255) & ~255; }
__host__ __device__ constexpr int fw_xscales(int K, bool int4) { return (int4 ? K >> 6 : K >> 5) | 1; }
// where the widened rows begin
__host__ __device__ constexpr int64_t fw_xnarrow(int M, int K, bool int4)
{
    return ((int64_t)M * (fw_xrow(K) + 4 * (int64_t)fw_xscales(K, int4)) + 15) & ~(int64_t)15;
}
__host__ __device__ constexpr int64_t fw_xbytes(int M, int K, bool int4, bool wide)
{
    return fw_xnarrow(M, K, int4) + (wide ? (int64_t)M * fw_xwide(K) : 0);
}

template <int FORM, int W>
__device__ __forceinline__ void fw_load_x(uint32_t lds, const FewArgs &a, int wave, int lane)
{
    constexpr bool INT4 = FORM == FEW_INT4;
    const int KB = a.K >> 1, segs = KB >> 4, ns = INT4 ? a.K >> 6 : a.K >> 5;
    const int xrow = fw_xrow(a.K), xs = fw_xscales(a.K, INT4), nc = (xrow + 1023) >> 10, nd = (ns + 63) >> 6;
    for (int i = wave; i < a.M * nc; i += W) {
        const int r = i / nc, c = i % nc, u = 64 * c + lane;
        if (u < xrow >> 4) fw_dma16(lds + r * xrow + 1024 * c, (uint32_t)r * KB + 16 * min(u ^ (r & 15), segs - 1), a.xq);
    }
    for (int i = wave; i < a.M * nd; i += W) {
        const int r = i / nd, c = i % nd, g = 64 * c + lane;
        const uint32_t to = lds + a.M * xrow + 4 * (r * xs + 64 * c);
        if (g < ns) {
            if constexpr (INT4) fw_dma4(to, 4 * ((uint32_t)r * ns + g), a.xscale);
            else fw_dma1(to, (uint32_t)r * ns + g, a.xscale);
        }
    }
}

// Waits until at most `stages` stages of N loads each are in flight.
template <int N, int MOST>
__device__ __forceinline__ void fw_wait_stages(int stages)
{
    static_assert(MOST <= 4 && N * MOST <= 63, "the loads in flight are counted in 6 bits");
    if (MOST > 3 && stages == 4) fw_wait<(MOST > 3 ? 4 * N : 0)>();
    else if (MOST > 2 && stages == 3) fw_wait<(MOST > 2 ? 3 * N : 0)>();
    else if (MOST > 1 && stages == 2) fw_wait<(MOST > 1 ? 2 * N : 0)>();
    else if (MOST > 0 && stages == 1) fw_wait<N>();
    else fw_wait<0>();
}

// W = WN WK waves: WN sets of 16 RT rows, the lines of each taken in turn by WK
// waves.  XB > 0: X is kept whole in XB bytes of LDS (XW: and widened); 0: it goes
// through the ring, where the WN waves of the same lines share it.
template <int FORM, int RT, int CT, bool GATED, int WN, int WK, int DEPTH, int XB, bool XW>
__global__ __launch_bounds__(64 * WN * WK) void w4a4_few_kernel(FewArgs a)
{
    typedef FewTile<FORM> Tile;
    constexpr bool INT4 = FORM == FEW_INT4, XS = XB > 0;
    constexpr int W = WN * WK, NT = GATED ? RT / 2 : RT, KH = GATED ? 2 : 1;     // tiles of output channels, weight rows of each
    constexpr int XT = XS ? 0 : CT, NL = RT * Tile::kLoads + XT * (WN == 1 ? Tile::kLoads : 2);
    constexpr int XRING = DEPTH * WK * XT * Tile::kBytes, RING = XRING + DEPTH * W * RT * Tile::kBytes;
    constexpr int SUMS = W * RT * CT * 1024, FIRST = RING > SUMS ? RING : SUMS;
    constexpr int UPS = WN * RT;                           // tiles of weight rows: up rows (1024 bytes) and biases (256) of each
    constexpr int LDS = FIRST + UPS * 1280 + CT * 2048 + XB;
    static_assert(!XS || CT == 1, "few enough rows");
    static_assert(LDS <= 160 * 1024, "a compute unit's LDS");
    __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % WN, wk = wave / WN;
    const int j16 = lane & 15, b = lane >> 4;
    // blocks 8 apart (the same XCD) take the sets of rows of the same channels in turn
    int tile = blockIdx.x, m0 = 0;
    if (a.chunks > 1) {
        const int per = 8 * a.chunks, in = tile % per;
        tile = tile / per * 8 + in % 8;
        m0 = in / 8 * (16 * CT);
    }
    const int n0 = tile * (16 * NT * WN);
    if (n0 >= a.N) return;
    const int KB = a.K >> 1, segs = KB >> 4, stages = (segs + 7) >> 3;
    const int srow = INT4 ? 4 * (a.K >> 6) : a.K >> 5;   // bytes of a row's scales

    // row of the weight: tile t of set w, row r
    auto wrow = [&](int w, int t, int r) {
        const int n = min(n0 + 16 * (NT * w + (GATED ? t >> 1 : t)) + r, a.N - 1);
        return GATED && (t & 1) ? a.N + n : n;
    };
    FewRows wo[RT], xo[CT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j) wo[t].code[j] = (uint32_t)wrow(wn, t, 8 * j + (lane >> 3)) * KB;
        wo[t].scale = (uint32_t)wrow(wn, t, j16) * srow;
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
#pragma unroll
        for (int j = 0; j < 2; ++j) xo[c].code[j] = (uint32_t)min(m0 + 16 * c + 8 * j + (lane >> 3), a.M - 1) * KB;
        xo[c].scale = (uint32_t)min(m0 + 16 * c + j16, a.M - 1) * srow;
    }
    const uint32_t lds0 = fw_lds(lds);
    auto xtile = [&](int i, int c) { return (((i % DEPTH) * WK + wk) * XT + c) * Tile::kBytes; };
    auto wtile = [&](int i, int t) { return XRING + (((i % DEPTH) * W + wave) * RT + t) * Tile::kBytes; };
    auto issue = [&](int i) {
        const int st = wk + i * WK;
#pragma unroll
        for (int t = 0; t < RT; ++t) fw_issue<FORM>(lds0 + wtile(i, t), wo[t], a.wq, a.wscale, st, segs, lane);
#pragma unroll
        for (int c = 0; c < XT; ++c) fw_issue<FORM, WN>(lds0 + xtile(i, c), xo[c], a.xq, a.xscale, st, segs, lane, wn);
    };
    const int mine = wk < stages ? (stages - wk + WK - 1) / WK : 0;

    f32x4 acc[RT][CT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    // the epilogue's operands, ahead of the stages: other waves read them, so a wave
    // waits for its share before the sums' barrier, whether it has a stage or not
    uint8_t *epi_up = lds + FIRST, *epi_bias = epi_up + UPS * 1024, *epi_h = epi_bias + UPS * 256;
    for (int u = wave; u < UPS + CT; u += W) {
        if (u < UPS) {
            const int w = u / RT, t = u % RT;
            fw_dma16(lds0 + FIRST + 1024 * u, (uint32_t)wrow(w, t, lane >> 2) * 64 + 16 * (lane & 3), a.up);
            if (a.bias) {
                const int n = min(n0 + 16 * (NT * w + (GATED ? t >> 1 : t)) + 2 * (lane & 7), a.N - 2);
                fw_dma4(lds0 + FIRST + 1024 * UPS + 256 * u, 2 * (uint32_t)(GATED && (t & 1) ? a.N + n : n), a.bias);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                fw_dma16(lds0 + FIRST + 1280 * UPS + 2048 * (u - UPS) + 1024 * j,
                         (uint32_t)min(m0 + 16 * (u - UPS) + 8 * j + (lane >> 3), a.M - 1) * 128 + 16 * (lane & 7), a.h);
        }
    }
    const uint8_t *xl = lds + LDS - XB;
    if constexpr (XS) fw_load_x<FORM, W>(lds0 + LDS - XB, a, wave, lane);
    // WN = 1: a wave's ring is its own, DEPTH stages ahead.  Else one barrier per
    // stage, and the place that a stage leaves is filled after the next one's.
    constexpr int AHEAD = WN == 1 ? DEPTH : DEPTH - 1;
    static_assert(AHEAD >= 1, "a stage is on its way before it is read");
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (i < mine) issue(i);
    const int xr = min(j16, a.M - 1), xrow = fw_xrow(a.K);
    const float *xls = reinterpret_cast<const float *>(xl + a.M * xrow) + xr * fw_xscales(a.K, INT4);
    static_assert(!XW || (XS && INT4), "only INT4 is widened");
    uint8_t *xw = lds + LDS - XB + (XW ? fw_xnarrow(a.M, a.K, INT4) : 0);
    const int xwide = fw_xwide(a.K);
    if constexpr (XS) {
        fw_wait_stages<NL, AHEAD>(min(AHEAD, mine));       // the wave's share of X has arrived
        __syncthreads();
        if constexpr (XW) {
            const int units = segs * 2;                    // of 8 code bytes
            for (int i = threadIdx.x; i < a.M * units; i += 64 * W) {
                const int r = i / units, u = i % units;
                long x0, x1;
                fw_widen(*reinterpret_cast<const uint2 *>(xl + r * xrow + 16 * ((u >> 1) ^ (r & 15)) + 8 * (u & 1)), x0, x1);
                long *o = reinterpret_cast<long *>(xw + r * xwide + 16 * (u ^ (r & 15)));
                o[0] = x0, o[1] = x1;
            }
            __syncthreads();
        }
    }
    // the lane's E8M0 byte for product s of a tile (in the low byte)
    auto e8m0 = [&](const uint8_t *tile, int s) {
        const uint8_t *p = tile + Tile::kCodes;
        if constexpr (FORM == FEW_MX) return (int)(*reinterpret_cast<const uint32_t *>(p + 64 * (b >> 1) + 4 * j16) >> (8 * (2 * (b & 1) + s)));
        else return *reinterpret_cast<const int *>(p + 256 * s + 4 * lane);
    };
    // the lane's 16-byte unit u of X, tile c
    auto xunit = [&](const uint8_t *S, int c, int st, int u) {
        return XS ? xl + xr * xrow + 16 * ((8 * st + u) ^ xr) : S + c * Tile::kBytes + j16 * 128 + 16 * fw_seg(j16, u);
    };
    const int rounds = WN == 1 ? mine : (stages + WK - 1) / WK;      // a barrier in each: the same for all waves
    for (int i = 0; i < rounds; ++i) {
        // this stage's loads are done: all but those of the stages after it
        fw_wait_stages<NL, AHEAD - 1>(min(AHEAD - 1, max(mine - 1 - i, 0)));
        if constexpr (WN > 1) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");     // every wave's, and the stage before is read
            if (i + AHEAD < mine) issue(i + AHEAD);
            if (i >= mine) continue;
        }
        const uint8_t *SX = lds + xtile(i, 0), *SW = lds + wtile(i, 0);
        const int st = wk + i * WK;
        if constexpr (INT4) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (4 * st + g >= (segs >> 1)) break;
                const int at = j16 * 128 + 16 * fw_seg(j16, 2 * g + (b >> 1)) + 8 * (b & 1);
                long x0[CT], x1[CT];
                float sx[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    if constexpr (XW) {
                        const long *x = reinterpret_cast<const long *>(xw + xr * xwide + 16 * ((4 * (4 * st + g) + b) ^ xr));
                        x0[c] = x[0], x1[c] = x[1];
                    } else {
                        fw_widen(*reinterpret_cast<const uint2 *>(xunit(SX, c, st, 2 * g + (b >> 1)) + 8 * (b & 1)), x0[c], x1[c]);
                    }
                    sx[c] = XS ? xls[4 * st + g]
                               : *reinterpret_cast<const float *>(SX + c * Tile::kBytes + Tile::kCodes + 4 * (16 * g + j16));
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint8_t *p = SW + t * Tile::kBytes;
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
                    const uint4 v = *reinterpret_cast<const uint4 *>(xunit(SX, c, st, 2 * b + s));
                    x[c] = (i32x8){in ? (int)v.x : 0, in ? (int)v.y : 0, in ? (int)v.z : 0, in ? (int)v.w : 0, 0, 0, 0, 0};
                    ex[c] = XS ? __builtin_bit_cast(int, xls[min(8 * st + 2 * b + s, segs - 1)])
                               : e8m0(SX + c * Tile::kBytes, s);
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint8_t *p = SW + t * Tile::kBytes;
                    const uint4 v = *reinterpret_cast<const uint4 *>(p + at);
                    const i32x8 w = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
                    const int ew = e8m0(p, s);
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        acc[t][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x[c], acc[t][c], 4, 4, 0, ew, 0, ex[c]);
                }
            }
        }
        if (WN == 1 && i + DEPTH < mine) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage has been read: its place is free
            issue(i + DEPTH);
        }
    }
    // the waves' sums: tile (t, c) of wave w at (w RT + t) CT + c.  The compiler does
    // not know of the loads to LDS: a wave without a stage has not waited for its
    // operands of the epilogue yet (one that had a stage has nothing under way)
    f32x4 *sums = reinterpret_cast<f32x4 *>(lds);
    fw_wait<0>();
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) sums[64 * ((wave * RT + t) * CT + c) + lane] = acc[t][c];
    __syncthreads();
    // a wave finishes one output tile after the other: lane (j16, b) has channels 4 b
    // .. 4 b + 3 of row j16
    for (int u = wave; u < WN * NT * CT; u += W) {
        const int c = u % CT, nt = u / CT, w = nt / NT;
        bf16x8 hhi, hlo;
        split_h(reinterpret_cast<const float *>(epi_h + 2048 * c + 128 * j16 + 32 * b), hhi, hlo);
        f32x4 y[KH];
#pragma unroll
        for (int k = 0; k < KH; ++k) {
            const int t = GATED ? 2 * (nt % NT) + k : nt % NT;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int g = 0; g < WK; ++g) v += sums[64 * (((g * WN + w) * RT + t) * CT + c) + lane];
            if (INT4) v *= 262144.0f;
            const bf16x8 ua = *reinterpret_cast<const bf16x8 *>(epi_up + 1024 * (w * RT + t) + 64 * j16 + 16 * b);
            v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ua, hhi, v, 0, 0, 0);
            v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ua, hlo, v, 0, 0, 0);
            if (a.bias) {
                const uint2 bi = *reinterpret_cast<const uint2 *>(epi_bias + 256 * (w * RT + t) + 8 * b);
                v[0] += bf16_to_f32(bi.x & 0xFFFFu), v[1] += bf16_to_f32(bi.x >> 16);
                v[2] += bf16_to_f32(bi.y & 0xFFFFu), v[3] += bf16_to_f32(bi.y >> 16);
            }
            y[k] = v;
        }
        const int m = m0 + 16 * c + j16, n = n0 + 16 * nt + 4 * b;
        if (m >= a.M || n >= a.N) continue;
        f32x4 o = y[0];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (a.act == FEW_GELU) o[k] = gelu_tanh(o[k]);
            else if (a.act == FEW_SILU) o[k] = silu(o[k]);
            if (GATED) o[k] *= y[KH - 1][k];
        }
        *reinterpret_cast<uint2 *>(a.Y + (size_t)m * a.N + n) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
}

// Launches WN WK waves per block of RTN tiles of channels each, with as many
// stages in flight as LDS and the count of loads take, up to DEPTHS.
template <int FORM, int CT, bool GATED, int WN, int WK, int RTN, int DEPTHS, int XB, bool XW = false>
void few_launch(const FewArgs &a, hipStream_t stream)
{
    typedef FewTile<FORM> Tile;
    constexpr int RT = RTN * (GATED ? 2 : 1), W = WN * WK, XT = XB ? 0 : CT;
    constexpr int STAGE = (WK * XT + W * RT) * Tile::kBytes, LOADS = RT * Tile::kLoads + XT * (WN == 1 ? Tile::kLoads : 2);
    constexpr int ROOM = (160 * 1024 - XB - WN * RT * 1280 - CT * 2048) / STAGE;
    constexpr int LEAST = ROOM < 63 / LOADS ? ROOM : 63 / LOADS, DEPTH = DEPTHS < LEAST ? DEPTHS : LEAST;
    if constexpr (WN > 1 && DEPTH < (WK > 2 ? 3 : 2)) {
        few_launch<FORM, CT, GATED, WN, WK / 2, RTN, DEPTHS, XB, XW>(a, stream);
    } else {
        const uint32_t tiles = (uint32_t)((a.N + 16 * RTN * WN - 1) / (16 * RTN * WN));
        const uint32_t grid = a.chunks > 1 ? (tiles + 7) / 8 * 8 * a.chunks : tiles;
        w4a4_few_kernel<FORM, RT, CT, GATED, WN, WK, DEPTH, XB, XW><<<grid, 64 * W, 0, stream>>>(a);
    }
}

// X in the ring.  The fewer tiles of 16 channels per compute unit, the fewer of
// them a block takes; the more, the more share the lines of X that come from the
// L2 (48 rows, us, one tile of channels per block / two / four: 28672 channels of
// 4096, MXFP4 35 / 28 / 23, INT4 46 / 44 / 42; 6144 channels 11 / 8.4 / 11 and 14
// / 12 / 21; 4096 of 14336 15 / 19 / 28 and 20 / 33 / 62).  INT4 with three or four
// tiles of rows is held by the widening, which eight waves of a tile share
// (2 x 6912 channels, 64 rows: 22 us, two tiles per block 25).
template <int FORM, int CT, bool GATED>
void few_ring(const FewArgs &a, hipStream_t stream)
{
    constexpr bool INT4 = FORM == FEW_INT4;
    const int64_t tiles = (a.N + 15) / 16, cus = device_cu_count();
    if (tiles > 3 * cus) few_launch<FORM, CT, GATED, 2, 2, 2, 4, 0>(a, stream);
    else if (tiles > cus && !(INT4 && CT > 2)) few_launch<FORM, CT, GATED, 2, 4, 1, 3, 0>(a, stream);
    else few_launch<FORM, CT, GATED, 1, INT4 ? 8 : 4, 1, INT4 ? 2 : 4, 0>(a, stream);
}

// X whole in LDS: up to a block per compute unit eight waves per tile, else four
// and more blocks (one row, us, four / eight waves: 4096 channels of 14336 INT4
// 13.8 / 10.4; 2 x 14336 of 4096 INT4 17.5 / 24.8, MXFP4 13.5 / 18.1).
template <int FORM, bool GATED, int XB, bool XW>
void few_whole(const FewArgs &a, hipStream_t stream)
{
    if ((a.N + 15) / 16 <= device_cu_count()) few_launch<FORM, 1, GATED, 1, 8, 1, 2, XB, XW>(a, stream);
    else few_launch<FORM, 1, GATED, 1, 4, 1, 2, XB, XW>(a, stream);
}

template <int FORM, bool GATED>
void few_rows(FewArgs a, hipStream_t stream)
{
    // more than 64 rows in equal sets of whole tiles
    a.chunks = (a.M + 63) / 64;
    const int rows = (a.M + a.chunks - 1) / a.chunks;
    // whole where it takes no more LDS than the ring's places for it would, and
    // widened where that fits too (INT4, one row / two, us: 6144 channels of 4096
    // 6.8 / 7.1, not widened 7.3 / 7.5; 28672 channels 16.2 / 16.5 and 17.3 / 17.5)
    constexpr bool INT4 = FORM == FEW_INT4;
    const int64_t x = fw_xbytes(a.M, a.K, INT4, false), wide = fw_xbytes(a.M, a.K, INT4, INT4);
    if (INT4 && rows <= 16 && wide <= 8192) few_whole<FORM, GATED, 8192, INT4>(a, stream);
    else if (INT4 && rows <= 16 && wide <= 17408) few_whole<FORM, GATED, 17408, INT4>(a, stream);
    else if (rows <= 16 && x <= 8192) few_whole<FORM, GATED, 8192, false>(a, stream);
    else if (rows <= 16 && x <= 17408) few_whole<FORM, GATED, 17408, false>(a, stream);
    else if (rows <= 16) few_ring<FORM, 1, GATED>(a, stream);
    else if (rows <= 32) few_ring<FORM, 2, GATED>(a, stream);
    else if (rows <= 48) few_ring<FORM, 3, GATED>(a, stream);
    else few_ring<FORM, 4, GATED>(a, stream);
}

template <bool GATED>
void few(const FewArgs &a, svdq_precision prec, hipStream_t stream)
{
    if (prec == SVDQ_INT4) few_rows<FEW_INT4, GATED>(a, stream);
    else if (a.K % 128 == 0) few_rows<FEW_MX, GATED>(a, stream);
    else few_rows<FEW_MX_ODD, GATED>(a, stream);
}

}  // namespace

hipError_t launch_w4a4_few(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                           const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N, int K,
                           svdq_precision prec, svdq_epilogue epi, uint16_t *Y, hipStream_t stream)
{
    const FewArgs a{xq, wq, xscale, wscale, h, up, bias, Y, M, N, K, epi == SVDQ_EPI_GELU_TANH ? FEW_GELU : FEW_NONE, 1};
    few<false>(a, prec, stream);
    return hipGetLastError();
}

hipError_t launch_w4a4_few_gated(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                                 const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N, int K,
                                 svdq_precision prec, svdq_activation act, uint16_t *Y, hipStream_t stream)
{
    const FewArgs a{xq, wq, xscale, wscale, h, up, bias, Y, M, N, K, act == SVDQ_ACT_GELU_TANH ? FEW_GELU : FEW_SILU, 1};
    few<true>(a, prec, stream);
    return hipGetLastError();
}

}  // namespace svdq
