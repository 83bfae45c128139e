// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//   Y_m = base_m + s_a (X_m A_a^T) B_a^T,   a = adapter of row m (none: Y_m = base_m)
//
// A plan (built once per step, used by every projection of the step) lists
// the rows adapter by adapter in tiles of at most 64 rows of one adapter; the
// rows without an adapter form the last tiles (adapter -1).
//
// Two kernels, both bound by HBM (rank 64 does 2 R (K + N) / (2 K + 4 N)
// operations per byte: 32 for N >> K, 37 at 4096 -> 12288, 43 at N = K; the
// second product runs twice, with the high and the low part of h; the chip's
// ratio is about 240):
//   down  a block takes one tile and one slice of K.  X and A_a go to LDS by
//         DMA in stages of 128 channels, three stages ahead of the products;
//         the four waves multiply a quarter of a stage each and add their fp32
//         sums in wave order at the end.  With one slice the block writes h =
//         s_a X A_a^T as a bf16 high and low part (together at least 16 bits of
//         significand, as the shared projection's own rank-32 branch does);
//         with more (few rows, so that the chip is filled) it writes the
//         slice's fp32 sums, and the second kernel adds them in slice order,
//         scales and splits.
//   up    a block takes one tile and 128 output channels, or up to eight times
//         128 in turn; the products with B_a accumulate in fp32, base is added
//         in fp32 and the row is rounded once.
// 9216 rows, 4096 -> 12288, rank 64: 118 us for 533 MB = 4.5 TB/s, where a copy
// of that size reaches 5.4 TB/s (128 channels per block: 139 us); rank 128: 140
// us.  16 rows of 16 adapters, 4096 -> 4096, rank 16: 4.3 + 4.2 us, latencies of
// the dependent loads (plan, rows, operands) and of two launches.  K and the
// widths are divided for the most tiles that rows and pool allow (the tiles in
// use are known on the device alone): 256 rows of one adapter take 9.5 us with a
// pool of 1 and 19.8 with one of 256.
// The order of every sum depends on the sizes alone, so results do not depend
// on which rows share a tile.
#include "svdq_internal.h"
#include "svdq_quant.h"

namespace svdq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int LR_ROWS = 64;            // rows per tile
constexpr int LR_PLAN_THREADS = 1024;
constexpr int LR_HEADER = 16;          // words: M, adapters, tiles

__device__ __forceinline__ uint32_t lr_pack2(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// s v as high and low bf16 parts of 8 channels.
__device__ __forceinline__ void lr_split(const float (&v)[8], float s, uint4 &hi, uint4 &lo)
{
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = v[2 * i] * s, y = v[2 * i + 1] * s;
        a[i] = lr_pack2(x, y);
        b[i] = lr_pack2(x - bits_f32(a[i] << 16), y - bits_f32(a[i] & 0xFFFF0000u));
    }
    hi = make_uint4(a[0], a[1], a[2], a[3]), lo = make_uint4(b[0], b[1], b[2], b[3]);
}

// ------------------------------------------------------------------- plan
//
// Words: header, then the tiles (adapter, rows, 0, 0), then 64 row numbers
// per tile; a tile of fewer rows repeats its first one.  A block knows its
// tile's rows from its own number alone, so their load does not wait for the
// tile's.

__host__ __device__ inline int64_t lr_max_tiles(int64_t M, int64_t n)
{
    const int64_t t = M / LR_ROWS + n + 1;
    return t < M ? t : M;
}

__global__ __launch_bounds__(LR_PLAN_THREADS) void lora_plan_kernel(const int32_t *__restrict__ index, int M, int n,
                                                                    int32_t *__restrict__ plan)
{
    __shared__ int count[kLoraMaxAdapters + 1];       // rows, then the next free place, of every bucket
    __shared__ int scan_tiles[LR_PLAN_THREADS];
    const int tid = threadIdx.x, lane = tid & 63;
    int4 *tiles = reinterpret_cast<int4 *>(plan + LR_HEADER);
    int32_t *place = plan + LR_HEADER + 4 * lr_max_tiles(M, n);
    for (int i = tid; i <= n; i += LR_PLAN_THREADS) count[i] = 0;
    __syncthreads();
    // bucket n holds the rows without an adapter; a wave whose rows share a
    // bucket (requests are runs of rows) takes one atomic for all of them
    const int rounds = (M + LR_PLAN_THREADS - 1) / LR_PLAN_THREADS;
    for (int r = 0; r < rounds; ++r) {
        const int m = r * LR_PLAN_THREADS + tid;
        int b = -1;
        if (m < M) b = index[m], b = (uint32_t)b < (uint32_t)n ? b : n;
        const int first = __builtin_amdgcn_readfirstlane(b);
        const uint64_t same = __ballot(b == first), in = __ballot(b >= 0);
        if (same == in) {
            if (lane == 0 && first >= 0) atomicAdd(&count[first], __popcll(in));
        } else if (b >= 0) {
            atomicAdd(&count[b], 1);
        }
    }
    __syncthreads();
    // exclusive sum of the tiles over the buckets, a few per thread
    const int per = n / LR_PLAN_THREADS + 1;
    const int b0 = tid * per;
    int nt = 0;
    for (int b = b0; b < b0 + per && b <= n; ++b) nt += (count[b] + LR_ROWS - 1) / LR_ROWS;
    scan_tiles[tid] = nt;
    __syncthreads();
    for (int d = 1; d < LR_PLAN_THREADS; d <<= 1) {
        const int c = tid >= d ? scan_tiles[tid - d] : 0;
        __syncthreads();
        scan_tiles[tid] += c;
        __syncthreads();
    }
    int t = scan_tiles[tid] - nt;
    for (int b = b0; b < b0 + per && b <= n; ++b) {
        const int c = count[b];
        count[b] = t * LR_ROWS;
        for (int r = 0; r < c; r += LR_ROWS)
            tiles[t++] = make_int4(b < n ? b : -1, c - r < LR_ROWS ? c - r : LR_ROWS, 0, 0);
    }
    if (tid == LR_PLAN_THREADS - 1) plan[0] = M, plan[1] = n, plan[2] = scan_tiles[tid];
    __syncthreads();                                 // orders the block's writes of the plan before its reads below
    for (int r = 0; r < rounds; ++r) {
        const int m = r * LR_PLAN_THREADS + tid;
        int b = -1;
        if (m < M) b = index[m], b = (uint32_t)b < (uint32_t)n ? b : n;
        const int first = __builtin_amdgcn_readfirstlane(b);
        const uint64_t same = __ballot(b == first), in = __ballot(b >= 0);
        if (same == in) {
            int p = 0;
            if (lane == 0 && first >= 0) p = atomicAdd(&count[first], __popcll(in));
            p = __builtin_amdgcn_readfirstlane(p);
            if (b >= 0) place[p + __popcll(in & ((1ull << lane) - 1))] = m;
        } else if (b >= 0) {
            place[atomicAdd(&count[b], 1)] = m;
        }
        __syncthreads();                             // keeps the places of a bucket close to row order
    }
    for (int e = tid; e < plan[2] * LR_ROWS; e += LR_PLAN_THREADS)
        if (e % LR_ROWS >= tiles[e / LR_ROWS].y) place[e] = place[e / LR_ROWS * LR_ROWS];
}

// ------------------------------------------------------------------- down

// Tile t of the plan; false past the last tile or for a plan of other sizes.
__device__ __forceinline__ bool lr_tile(const int32_t *plan, int M, int n, int t, int &adapter, int &count)
{
    if (plan[0] != M || plan[1] != n || t >= plan[2]) return false;
    const int2 v = *reinterpret_cast<const int2 *>(plan + LR_HEADER + 4 * (size_t)t);
    adapter = v.x, count = v.y;
    return true;
}

__device__ __forceinline__ const int32_t *lr_rows(const int32_t *plan, int M, int n, int t)
{
    return plan + LR_HEADER + 4 * lr_max_tiles(M, n) + (size_t)LR_ROWS * t;
}

typedef __attribute__((address_space(3))) uint8_t lr_lds_u8;
__device__ __forceinline__ uint32_t lr_lds_offset(const void *p)
{
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lr_lds_u8 *)p);
}

// One LDS-DMA load per lane: 16 bytes from sbase + voff to LDS lds + 16 lane.
// M0 is saved and restored around it.
__device__ __forceinline__ void lr_dma_b128(uint32_t lds, uint32_t voff, const void *sbase)
{
    uint32_t keep;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
                 : "=&s"(keep) : "s"(lds), "v"(voff), "s"(sbase) : "memory");
}

// A stage holds 128 channels (256 bytes) of the tile's rows of X and of A_a's
// rows.  16-byte segment s of LDS row r lies at s ^ (r % 16), so that the
// fragment reads of 16 consecutive rows hit different banks.
constexpr int LR_STAGE_K = 128;
constexpr int lr_stages(int NT) { return NT <= 4 ? 4 : 3; }
constexpr int lr_stage_bytes(int NT) { return (LR_ROWS + 16 * NT) * 2 * LR_STAGE_K; }

// The block's part of X A_a^T over stages st0 .. st1 - 1: G groups of 16 rows,
// NT tiles of 16 columns.  The loads (16 lanes per row: whole lines; loads in
// operand order, one row per lane, took four times the L1's cycles) run
// S - 1 stages ahead; every stage issues the same number of them, so the wait
// for a stage is a count.  Wave w multiplies channels 32 w .. + 31 of a stage.
// Rows past the tile repeat one of it and columns past R the last one: neither
// is used.  Past K both operands repeat the last channels and A's are zeroed.
template <int NT, int G>
__device__ __forceinline__ void lr_down(f32x4 (&acc)[4][NT], uint8_t *lds, const uint16_t *X, const uint16_t *a0,
                                        const int32_t *rows, int K, int R, int st0, int st1, int wave, int lane)
{
    constexpr int S = lr_stages(NT), XL = G, AL = NT;         // loads per wave and stage
    const int i16 = lane & 15, kb = lane >> 4;
    uint32_t xoff[XL], aoff[AL];
    // load q of the wave fills LDS rows 16 q + 4 w .. + 3, lane / 16 the row, lane % 16 the slot
    const int r4 = 4 * wave + kb;                             // row % 16
    const uint32_t sg = 16u * (uint32_t)(i16 ^ r4);
#pragma unroll
    for (int q = 0; q < XL; ++q) xoff[q] = (uint32_t)rows[16 * q + r4] * 2u * (uint32_t)K;
#pragma unroll
    for (int q = 0; q < AL; ++q) aoff[q] = (uint32_t)min(16 * q + r4, R - 1) * 2u * (uint32_t)K;
    auto issue = [&](int st) {
        const uint32_t k = min((uint32_t)min(st, st1 - 1) * 2u * LR_STAGE_K + sg, 2u * (uint32_t)K - 16u);
        uint8_t *b = lds + (st - st0) % S * lr_stage_bytes(NT) + 1024 * wave;
#pragma unroll
        for (int q = 0; q < XL; ++q) lr_dma_b128(lr_lds_offset(b + 4096 * q), xoff[q] + k, X);
#pragma unroll
        for (int q = 0; q < AL; ++q) lr_dma_b128(lr_lds_offset(b + 4096 * (4 + q)), aoff[q] + k, a0);
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(st0 + i);
    for (int st = st0; st < st1; ++st) {
        // this wave's loads of the stage have landed and its reads of the stage
        // before, which the next loads overwrite, are complete; after the
        // barrier all waves' are
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S - 2) * (XL + AL)) : "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(st + S - 1);
        const uint8_t *b = lds + (st - st0) % S * lr_stage_bytes(NT) + 16 * ((4 * wave + kb) ^ i16) + 256 * i16;
        bf16x8 x[G], a[NT];
#pragma unroll
        for (int g = 0; g < G; ++g) x[g] = *reinterpret_cast<const bf16x8 *>(b + 4096 * g);
#pragma unroll
        for (int j = 0; j < NT; ++j) a[j] = *reinterpret_cast<const bf16x8 *>(b + 4096 * (4 + j));
        if ((st + 1) * LR_STAGE_K > K && st * LR_STAGE_K + 32 * wave + 8 * kb >= K) {
#pragma unroll
            for (int j = 0; j < NT; ++j) a[j] = __builtin_bit_cast(bf16x8, make_uint4(0u, 0u, 0u, 0u));
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[g][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[g], a[j], acc[g][j], 0, 0, 0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// h of a tile is stored in the second kernel's operand order: for rows 16 g ..
// and channels 32 k .. of the tile, lane (row % 16, 8-channel part) has 8
// channels.  lr_h is the index of that lane in units of 8 channels; the
// channels past R are zeros.
__host__ __device__ constexpr int lr_ksteps(int NT) { return (NT + 1) / 2; }
__device__ __forceinline__ size_t lr_h(int KS, int t, int g, int k) { return ((size_t)(4 * (size_t)t + g) * KS + k) * 64; }

// One slice of K: h = s_a X A_a^T as bf16, the high parts of a lane's 8
// channels at 2 lr_h, the low parts 64 lanes on.  More: the slice's part of
// X A_a^T in fp32.  NT: 16-wide tiles of R.
template <int NT>
__global__ __launch_bounds__(256) void lora_down_kernel(
    const uint16_t *__restrict__ X, const uint16_t *__restrict__ A, const float *__restrict__ scale,
    const int32_t *__restrict__ plan, int M, int K, int R, int n, int slices, int stages_per_slice,
    float *__restrict__ work)
{
    constexpr int RS = 16 * NT + 4, KS = lr_ksteps(NT);
    static_assert(4 * LR_ROWS * RS * 4 <= lr_stages(NT) * lr_stage_bytes(NT), "the waves' sums reuse the stages");
    __shared__ __attribute__((aligned(16))) uint8_t lds[lr_stages(NT) * lr_stage_bytes(NT)];
    const int slice = blockIdx.x % slices, t = blockIdx.x / slices;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, kb = lane >> 4;
    int adapter, count;
    if (!lr_tile(plan, M, n, t, adapter, count) || adapter < 0) return;
    const int32_t *rows = lr_rows(plan, M, n, t);
    const int stages = (K + LR_STAGE_K - 1) / LR_STAGE_K;
    const int st0 = slice * stages_per_slice, st1 = min(stages, st0 + stages_per_slice);
    const uint16_t *a0 = A + (size_t)adapter * R * K;
    f32x4 acc[4][NT] = {};
    if (count <= 16) lr_down<NT, 1>(acc, lds, X, a0, rows, K, R, st0, st1, wave, lane);
    else lr_down<NT, 4>(acc, lds, X, a0, rows, K, R, st0, st1, wave, lane);
    // the waves' sums are added in wave order; a lane holds rows 4 kb + i,
    // column i16 of its tiles
    float (*red)[LR_ROWS][RS] = reinterpret_cast<float (*)[LR_ROWS][RS]>(lds);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        if (16 * g >= count) break;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[wave][16 * g + 4 * kb + i][16 * j + i16] = acc[g][j][i];
    }
    __syncthreads();
    const float s = scale[adapter];
    const size_t slice_lanes = lr_h(KS, (int)lr_max_tiles(M, n), 0, 0);
    for (int e = threadIdx.x; e < (count <= 16 ? 1 : 4) * KS * 64; e += 256) {
        const int l = e & 63, k = (e >> 6) % KS, g = (e >> 6) / KS;
        const int p = 16 * g + (l & 15), r = 32 * k + 8 * (l >> 4);
        float v[8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            f32x4 u = {};
            if (r < R && p < count) {
                u = *reinterpret_cast<const f32x4 *>(&red[0][p][r + 4 * q]);
#pragma unroll
                for (int w = 1; w < 4; ++w) u += *reinterpret_cast<const f32x4 *>(&red[w][p][r + 4 * q]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * q + i] = u[i];
        }
        if (slices == 1) {
            uint4 *o = (uint4 *)work + 2 * lr_h(KS, t, g, k) + l;
            lr_split(v, s, o[0], o[64]);
        } else {
            f32x4 *o = (f32x4 *)work + 2 * (slice * slice_lanes + lr_h(KS, t, g, k) + l);
            o[0] = (f32x4){v[0], v[1], v[2], v[3]}, o[1] = (f32x4){v[4], v[5], v[6], v[7]};
        }
    }
}

// --------------------------------------------------------------------- up
//
// A block takes one tile and `width` output channels, 128 at a time, base's and
// B_a's next 128 on their way during the products.  Wave g multiplies rows 16 g
// .. of the tile with all 128: product tile j has the channels 8 i + j (i = 0 ..
// 15), so a lane's sums are 8 consecutive channels of four rows and base and Y
// move as 256 bytes per row and instruction.  B_a's rows go through LDS, once
// for the four waves.  A tile of at most 16 rows is shared out by channels
// instead, 32 per wave, B_a straight from memory.
constexpr int LR_UP_N = 128;

template <int KS>
__device__ __forceinline__ void lr_load_h(bf16x8 (&hi)[KS], bf16x8 (&lo)[KS], const float *work, int t, int g,
                                          int slices, size_t slice_lanes, float s_a, int lane)
{
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        uint4 a, b;
        if (slices == 1) {
            const uint4 *p = (const uint4 *)work + 2 * lr_h(KS, t, g, k) + lane;
            a = p[0], b = p[64];
        } else {
            const f32x4 *p = (const f32x4 *)work + 2 * (lr_h(KS, t, g, k) + lane);
            f32x4 u = p[0], v = p[1];
            int q = 1;
            for (; q + 3 < slices; q += 4) {             // four slices' loads in flight, added in slice order
                f32x4 x[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i][0] = p[2 * (q + i) * slice_lanes], x[i][1] = p[2 * (q + i) * slice_lanes + 1];
#pragma unroll
                for (int i = 0; i < 4; ++i) u += x[i][0], v += x[i][1];
            }
            for (; q < slices; ++q) u += p[2 * q * slice_lanes], v += p[2 * q * slice_lanes + 1];
            const float f[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
            lr_split(f, s_a, a, b);
        }
        hi[k] = __builtin_bit_cast(bf16x8, a), lo[k] = __builtin_bit_cast(bf16x8, b);
    }
}

// KS: 32-wide steps of R.
template <int KS>
__global__ __launch_bounds__(256) void lora_up_kernel(const float *__restrict__ work, const uint16_t *__restrict__ B,
                                                      const float *__restrict__ scale,
                                                      const int32_t *__restrict__ plan, int M, int N, int R, int n,
                                                      int slices, int nblocks, int width, const uint16_t *base, uint16_t *Y)
{
    constexpr int BS = 32 * KS + 8;                      // LDS row: B_a's channels, zeros up to 32 KS, 16 B pad
    __shared__ __attribute__((aligned(16))) uint16_t bs[LR_UP_N * BS];
    const int t = blockIdx.x / nblocks, n_first = (blockIdx.x % nblocks) * width, n_end = min(N, n_first + width);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int i16 = lane & 15, kb = lane >> 4;
    int adapter, count;
    if (!lr_tile(plan, M, n, t, adapter, count)) return;
    const int32_t *rows = lr_rows(plan, M, n, t);
    if (adapter < 0) {                                   // rows without an adapter: copied, unless in place
        if (Y == base) return;
        for (int c = n_first + 8 * i16; c < n_end; c += LR_UP_N)
            for (int p = tid >> 4; p < count; p += 16) {
                const size_t o = (size_t)rows[p] * N + c;
                *reinterpret_cast<uint4 *>(Y + o) = *reinterpret_cast<const uint4 *>(base + o);
            }
        return;
    }
    const uint16_t *ba = B + (size_t)adapter * N * R;
    const float s_a = scale[adapter];
    const size_t slice_lanes = lr_h(KS, (int)lr_max_tiles(M, n), 0, 0);
    bf16x8 hi[KS], lo[KS];
    if (count <= 16) {
        lr_load_h<KS>(hi, lo, work, t, 0, slices, slice_lanes, s_a, lane);
        const int4 row = *reinterpret_cast<const int4 *>(rows + 4 * kb);
        for (int n0 = n_first + 32 * wave; n0 < n_end; n0 += LR_UP_N) {
            // channels n0 + 2 i16 + j: two per lane
            const int c = n0 + 2 * i16, cc = min(c, N - 2);
            const size_t off[4] = {(size_t)row.x * N + cc, (size_t)row.y * N + cc, (size_t)row.z * N + cc, (size_t)row.w * N + cc};
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const uint32_t *>(base + off[i]);
            uint4 b[KS][2];
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j)              // chunks past R repeat the last one and meet zeros of h
                    b[k][j] = *reinterpret_cast<const uint4 *>(ba + (size_t)(cc + j) * R + min(32 * k + 8 * kb, R - 8));
            f32x4 acc[2] = {};
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bf16x8 bb = __builtin_bit_cast(bf16x8, b[k][j]);
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[k], bb, acc[j], 0, 0, 0);
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[k], bb, acc[j], 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * kb + i < count && c < N)
                    *reinterpret_cast<uint32_t *>(Y + off[i]) =
                        lr_pack2(bits_f32(y[i] << 16) + acc[0][i], bits_f32(y[i] & 0xFFFF0000u) + acc[1][i]);
        }
        return;
    }
    // channels n0 + 8 i16 .. + 7 of rows 16 wave + 4 kb + i
    const int4 row = *reinterpret_cast<const int4 *>(rows + 16 * wave + 4 * kb);
    const size_t off[4] = {(size_t)row.x * N, (size_t)row.y * N, (size_t)row.z * N, (size_t)row.w * N};
    // LDS row 16 j + i holds channel 8 i + j
    constexpr int CH = 4 * KS, ST = LR_UP_N * CH / 256;  // 16-byte chunks of an LDS row, of a thread
    u32x4 y[4], st[ST];
    auto load = [&](u32x4 (&y)[4], u32x4 (&st)[ST], int n0) {
        const int cc = min(n0 + 8 * i16, N - 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const u32x4 *>(base + off[i] + cc);
#pragma unroll
        for (int q = 0; q < ST; ++q) {
            const int e = tid + 256 * q, ch = e % CH, nn = min(n0 + e / CH, N - 1);
            st[q] = *reinterpret_cast<const u32x4 *>(ba + (size_t)nn * R + min(8 * ch, R - 8));
        }
    };
    load(y, st, n_first);
    lr_load_h<KS>(hi, lo, work, t, wave, slices, slice_lanes, s_a, lane);
    for (int n0 = n_first;; n0 += LR_UP_N) {
#pragma unroll
        for (int q = 0; q < ST; ++q) {
            const int e = tid + 256 * q, ch = e % CH, nn = e / CH;
            *reinterpret_cast<u32x4 *>(&bs[(16 * (nn & 7) + (nn >> 3)) * BS + 8 * ch]) = st[q];
        }
        const bool more = n0 + LR_UP_N < n_end;
        u32x4 y2[4], st2[ST];
        load(y2, st2, more ? n0 + LR_UP_N : n0);         // on their way during the products
        __syncthreads();
        f32x4 acc[8] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bf16x8 b = *reinterpret_cast<const bf16x8 *>(&bs[(16 * j + i16) * BS + 32 * k + 8 * kb]);
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi[k], b, acc[j], 0, 0, 0);
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[k], b, acc[j], 0, 0, 0);
            }
        const int c = n0 + 8 * i16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (16 * wave + 4 * kb + i >= count || c >= N) continue;
            const uint32_t w[4] = {y[i][0], y[i][1], y[i][2], y[i][3]};
            uint32_t v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] = lr_pack2(bits_f32(w[q] << 16) + acc[2 * q][i], bits_f32(w[q] & 0xFFFF0000u) + acc[2 * q + 1][i]);
            *reinterpret_cast<uint4 *>(Y + off[i] + c) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        if (!more) break;
        __syncthreads();                                 // all have read B_a's channels
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = y2[i];
#pragma unroll
        for (int q = 0; q < ST; ++q) st[q] = st2[q];
    }
}

// Slices of K, in stages of 128 channels: enough blocks for the chip, at
// least two stages each, at most four: more shorten the first kernel less than
// they lengthen the second, which adds them up (16 rows of 16 adapters, 4096
// -> 4096, rank 16: 11.2 us with one slice, 8.3 with 4, 9.1 with 16; 1111 rows
// of 7, 2048 -> 6144, rank 32: 15.5, 13.8 and 14.7 us).
constexpr int LR_MAX_SLICES = 4;

int lr_slices(int64_t M, int K, int n, int &stages_per_slice)
{
    const int64_t tiles = lr_max_tiles(M, n);
    const int stages = (K + LR_STAGE_K - 1) / LR_STAGE_K;
    int64_t s = device_cu_count() / tiles;
    s = s > LR_MAX_SLICES ? LR_MAX_SLICES : s;
    s = s > stages / 2 ? stages / 2 : s;
    s = s < 1 ? 1 : s;
    stages_per_slice = (int)((stages + s - 1) / s);
    return (stages + stages_per_slice - 1) / stages_per_slice;
}

// 32-wide steps of R that the kernels hold: 1, 2 or 4.
int lr_rank_steps(int R) { return R <= 32 ? 1 : (R <= 64 ? 2 : 4); }

}  // namespace

size_t lora_plan_size(int M, int n) { return 4 * (size_t)(LR_HEADER + (4 + LR_ROWS) * lr_max_tiles(M, n)); }

size_t lora_work_bytes(int M, int K, int R, int n)
{
    int per;
    return (size_t)lr_slices(M, K, n, per) * LR_ROWS * lr_max_tiles(M, n) * 32 * lr_rank_steps(R) * sizeof(float);
}

hipError_t launch_lora_plan(const int32_t *index, int M, int n, void *plan, hipStream_t stream)
{
    lora_plan_kernel<<<1, LR_PLAN_THREADS, 0, stream>>>(index, M, n, (int32_t *)plan);
    return hipGetLastError();
}

hipError_t launch_lora_linear(const uint16_t *X, const uint16_t *A, const uint16_t *B, const float *scale,
                              const void *plan, const uint16_t *base, int M, int N, int K, int R, int n, uint16_t *Y,
                              float *work, hipStream_t stream)
{
    const int32_t *pl = (const int32_t *)plan;
    const int64_t tiles = lr_max_tiles(M, n);
    int per;
    const int slices = lr_slices(M, K, n, per);
    const dim3 grid((uint32_t)(tiles * slices));
#define LR_DOWN(NT) \
    lora_down_kernel<NT><<<grid, 256, 0, stream>>>(X, A, scale, pl, M, K, R, n, slices, per, work)
    if (R <= 16) LR_DOWN(1);
    else if (R <= 32) LR_DOWN(2);
    else if (R <= 64) LR_DOWN(4);
    else LR_DOWN(8);
#undef LR_DOWN
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // several times 128 channels per block, so that h is loaded once for them,
    // where at least four blocks per compute unit are left.  9216 rows, 4096 ->
    // 12288, rank 64: 1 x 139 us, 2 x 126, 4 x 118, 8 x 116 to 119; 13 of 96
    // parts, which leave uneven blocks, 128.
    const int64_t each = (N + LR_UP_N - 1) / LR_UP_N;
    const int64_t many = tiles * each / (4 * (int64_t)device_cu_count());      // blocks of 128 over the least number
    const int width = LR_UP_N * (int)(many < 1 ? 1 : (many > 8 ? 8 : many));
    const int nblocks = (N + width - 1) / width;
    const dim3 ugrid((uint32_t)(tiles * nblocks));
#define LR_UP(KS) \
    lora_up_kernel<KS><<<ugrid, 256, 0, stream>>>(work, B, scale, pl, M, N, R, n, slices, nblocks, width, base, Y)
    if (R <= 32) LR_UP(1);
    else if (R <= 64) LR_UP(2);
    else LR_UP(4);
#undef LR_UP
    return hipGetLastError();
}

}  // namespace svdq
