// lora.hip -- low-rank adapters of many requests beside a shared projection:
//
//   Y_m = base_m + s_a (X_m A_a^T) B_a^T,   a = adapter of row m (none: Y_m = base_m)
//
// A plan (built once per step, used by every projection of the step) lists
// the rows adapter by adapter in tiles of at most 64 rows of one adapter; the
// rows without an adapter form the last tiles (adapter -1).
//
// Two kernels, both bound by HBM:
//   down  a block takes one tile and one slice of K; its four waves take the
//         slice's 64-channel chunks in turn, so a chunk of A_a is read once
//         for up to 64 rows, and add their fp32 sums in wave order.  The
//         slices (few rows: many slices, so that the chip is filled) go to
//         the workspace as separate fp32 sums.
//   up    a block takes one tile and a run of output channels, adds the
//         slices in slice order, scales by s_a and splits h into a bf16 high
//         and low part (together 16 bits of significand, as the shared
//         projection's own rank-32 branch does); the products with B_a
//         accumulate in fp32, base is added in fp32 and the row is rounded
//         once.
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

constexpr int LR_ROWS = 64;            // rows per tile
constexpr int LR_PLAN_THREADS = 1024;
constexpr int LR_HEADER = 16;          // words: M, adapters, tiles
constexpr int LR_SLICE = 256;          // least channels per slice: one 64-channel chunk per wave

__device__ __forceinline__ uint32_t lr_pack2(float lo, float hi)
{
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// ------------------------------------------------------------------- plan
//
// Words: header, then the tiles (adapter, first place, rows, 0), then the row
// at every place.

__host__ __device__ inline int64_t lr_max_tiles(int64_t M, int64_t n)
{
    const int64_t t = M / LR_ROWS + n + 1;
    return t < M ? t : M;
}

__global__ __launch_bounds__(LR_PLAN_THREADS) void lora_plan_kernel(const int32_t *__restrict__ index, int M, int n,
                                                                    int32_t *__restrict__ plan)
{
    __shared__ int count[kLoraMaxAdapters + 1];       // rows, then the next free place, of every bucket
    __shared__ int scan_rows[LR_PLAN_THREADS], scan_tiles[LR_PLAN_THREADS];
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
    // exclusive sums of rows and tiles over the buckets, a few per thread
    const int per = n / LR_PLAN_THREADS + 1;
    const int b0 = tid * per;
    int rows = 0, nt = 0;
    for (int b = b0; b < b0 + per && b <= n; ++b) {
        rows += count[b];
        nt += (count[b] + LR_ROWS - 1) / LR_ROWS;
    }
    scan_rows[tid] = rows, scan_tiles[tid] = nt;
    __syncthreads();
    for (int d = 1; d < LR_PLAN_THREADS; d <<= 1) {
        const int a = tid >= d ? scan_rows[tid - d] : 0, c = tid >= d ? scan_tiles[tid - d] : 0;
        __syncthreads();
        scan_rows[tid] += a, scan_tiles[tid] += c;
        __syncthreads();
    }
    int at = scan_rows[tid] - rows, t = scan_tiles[tid] - nt;
    for (int b = b0; b < b0 + per && b <= n; ++b) {
        const int c = count[b];
        count[b] = at;
        for (int r = 0; r < c; r += LR_ROWS)
            tiles[t++] = make_int4(b < n ? b : -1, at + r, c - r < LR_ROWS ? c - r : LR_ROWS, 0);
        at += c;
    }
    if (tid == LR_PLAN_THREADS - 1) plan[0] = M, plan[1] = n, plan[2] = scan_tiles[tid];
    __syncthreads();
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
}

// ------------------------------------------------------------------- down

// Tile t of the plan; false past the last tile or for a plan of other sizes.
__device__ __forceinline__ bool lr_tile(const int32_t *plan, int M, int n, int t, int4 &tile, const int32_t *&rows)
{
    if (plan[0] != M || plan[1] != n || t >= plan[2]) return false;
    tile = reinterpret_cast<const int4 *>(plan + LR_HEADER)[t];
    rows = plan + LR_HEADER + 4 * lr_max_tiles(M, n) + tile.y;
    return true;
}

// work[slice][place][R] = the slice's part of X A_a^T.  NT: 16-wide tiles of R.
template <int NT>
__global__ __launch_bounds__(256) void lora_down_kernel(const uint16_t *__restrict__ X, const uint16_t *__restrict__ A,
                                                        const int32_t *__restrict__ plan, int M, int K, int R, int n,
                                                        int slices, int chunks_per_slice, float *__restrict__ work)
{
    __shared__ float red[LR_ROWS][16 * NT + 4];
    const int slice = blockIdx.x % slices;
    int4 tile;
    const int32_t *rows;
    if (!lr_tile(plan, M, n, blockIdx.x / slices, tile, rows) || tile.x < 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int i16 = lane & 15, kb = lane >> 4;
    const int groups = (tile.z + 15) >> 4;
    const int chunks = (K + 63) >> 6;
    const int c_end = min(chunks, (slice + 1) * chunks_per_slice);

    const uint16_t *xrow[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int p = min(16 * g + i16, tile.z - 1);       // rows past the tile repeat its last one, never stored
        xrow[g] = X + (size_t)rows[p] * K + 8 * kb;
    }
    const uint16_t *arow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        arow[j] = A + ((size_t)tile.x * R + min(16 * j + i16, R - 1)) * K + 8 * kb;   // columns past R: never stored

    f32x4 acc[4][NT] = {};
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int c = slice * chunks_per_slice + wave; c < c_end; c += 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = 64 * c + 32 * h;
            const bool in = k + 8 * kb < K;
            uint4 a[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) a[j] = in ? *reinterpret_cast<const uint4 *>(arow[j] + k) : zero;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (g < groups) {
                    const uint4 x = in ? *reinterpret_cast<const uint4 *>(xrow[g] + k) : zero;
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[g][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, a[j]), acc[g][j], 0, 0, 0);
                }
            }
        }
    }
    // the waves' sums in wave order; lane holds rows 4 kb + i, column i16
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (wave == w) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (g < groups)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float &d = red[16 * g + 4 * kb + i][16 * j + i16];
                            d = w == 0 ? acc[g][j][i] : d + acc[g][j][i];
                        }
        }
        __syncthreads();
    }
    float *out = work + ((size_t)slice * M + tile.y) * R;
    for (int e = threadIdx.x; e < tile.z * R; e += 256) out[e] = red[e / R][e % R];
}

// --------------------------------------------------------------------- up

// KS: 32-wide steps of the product's 2 R channels (h high, h low).
template <int KS>
__global__ __launch_bounds__(256) void lora_up_kernel(const float *__restrict__ work, const uint16_t *__restrict__ B,
                                                      const float *__restrict__ scale,
                                                      const int32_t *__restrict__ plan, int M, int N, int R, int n,
                                                      int slices, int nblocks, int nsteps, const uint16_t *base,
                                                      uint16_t *Y)
{
    constexpr int HS = 32 * KS + 8;                      // LDS row: high and low parts, zero up to 32 KS, 16 B pad
    __shared__ __attribute__((aligned(16))) uint16_t hs[LR_ROWS * HS];
    int4 tile;
    const int32_t *rows;
    if (!lr_tile(plan, M, n, blockIdx.x / nblocks, tile, rows)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int i16 = lane & 15, kb = lane >> 4;
    const int nb = blockIdx.x % nblocks;
    const int groups = (tile.z + 15) >> 4;
    if (tile.x < 0) {                                    // rows without an adapter: copied, unless in place
        if (Y == base) return;
        for (int s = 0; s < nsteps; ++s) {
            const int c = ((nb * nsteps + s) * 256) + 8 * (tid & 31);
            if (c >= N) continue;
            for (int p = tid >> 5; p < tile.z; p += 8) {
                const size_t o = (size_t)rows[p] * N + c;
                *reinterpret_cast<uint4 *>(Y + o) = *reinterpret_cast<const uint4 *>(base + o);
            }
        }
        return;
    }
    // h of the tile: slices in slice order, scaled, high and low bf16 parts
    const float s = scale[tile.x];
    const float *part = work + (size_t)tile.y * R;
    for (int e = tid; e < 16 * groups * 16 * KS; e += 256) {
        const int p = e / (16 * KS), r = e % (16 * KS);
        float v = 0.0f;
        if (p < tile.z && r < R) {
            v = part[(size_t)p * R + r];
            for (int q = 1; q < slices; ++q) v += part[((size_t)q * M + p) * R + r];
            v *= s;
        }
        const uint32_t hi = lr_pack2(v, 0.0f) & 0xFFFFu;
        const uint32_t lo = lr_pack2(v - bits_f32(hi << 16), 0.0f) & 0xFFFFu;
        if (r < R) {
            hs[p * HS + r] = (uint16_t)hi;
            hs[p * HS + R + r] = (uint16_t)lo;
        } else {                                         // 32 KS - 2 R zeros, two per r
            hs[p * HS + 2 * R + 2 * (r - R)] = 0;
            hs[p * HS + 2 * R + 2 * (r - R) + 1] = 0;
        }
    }
    __syncthreads();
    const int chunks = R >> 3;
    const uint16_t *ba = B + (size_t)tile.x * N * R;
    for (int st = 0; st < nsteps; ++st) {
        const int n0 = (nb * nsteps + st) * 256 + 64 * wave;
        if (n0 >= N) break;
        // base: 16 consecutive channels n0 + 16 kb .. of row 16 g + i16
        uint4 y[4][2];
        size_t off[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int p = 16 * g + i16;
            off[g] = (size_t)rows[min(p, tile.z - 1)] * N + n0 + 16 * kb;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (p < tile.z && n0 + 16 * kb + 8 * h < N)
                    y[g][h] = *reinterpret_cast<const uint4 *>(base + off[g] + 8 * h);
        }
        // A operand of tile j: row i is channel n0 + 16 (i / 4) + 4 j + i % 4,
        // so that a lane's four tiles hold 16 consecutive channels
        uint4 b[KS][4];
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            int c = 4 * k + kb;
            const bool in = c < 2 * chunks;
            c = c >= chunks ? c - chunks : c;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int nn = n0 + 16 * (i16 >> 2) + 4 * j + (i16 & 3);
                b[k][j] = in && nn < N ? *reinterpret_cast<const uint4 *>(ba + (size_t)nn * R + 8 * c)
                                       : make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            if (g >= groups) break;
            f32x4 acc[4] = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const bf16x8 h = *reinterpret_cast<const bf16x8 *>(&hs[(16 * g + i16) * HS + 32 * k + 8 * kb]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[k][j]), h, acc[j], 0,
                                                                     0, 0);
            }
            if (16 * g + i16 < tile.z) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (n0 + 16 * kb + 8 * h >= N) continue;
                    const uint32_t w[4] = {y[g][h].x, y[g][h].y, y[g][h].z, y[g][h].w};
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o[q] = lr_pack2(bits_f32(w[q] << 16) + acc[2 * h + (q >> 1)][2 * (q & 1)],
                                        bits_f32(w[q] & 0xFFFF0000u) + acc[2 * h + (q >> 1)][2 * (q & 1) + 1]);
                    *reinterpret_cast<uint4 *>(Y + off[g] + 8 * h) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
}

// Slices of K: enough blocks for the chip (the tiles are at least the rows'
// tiles; with more adapters than that, one per adapter), none below LR_SLICE.
int lr_slices(int64_t M, int K, int n, int &chunks_per_slice)
{
    const int64_t tiles = lr_max_tiles(M, n);
    const int chunks = (K + 63) / 64;
    int64_t s = (2 * (int64_t)device_cu_count() + tiles - 1) / tiles;
    const int64_t most = K / LR_SLICE > 1 ? K / LR_SLICE : 1;
    s = s < 1 ? 1 : (s > most ? most : s);
    chunks_per_slice = (int)((chunks + s - 1) / s);
    return (chunks + chunks_per_slice - 1) / chunks_per_slice;
}

}  // namespace

size_t lora_plan_size(int M, int n) { return 4 * (size_t)(LR_HEADER + 4 * lr_max_tiles(M, n) + M); }

size_t lora_work_bytes(int M, int K, int R, int n)
{
    int per;
    return (size_t)lr_slices(M, K, n, per) * M * R * sizeof(float);
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
#define LR_DOWN(NT) lora_down_kernel<NT><<<grid, 256, 0, stream>>>(X, A, pl, M, K, R, n, slices, per, work)
    if (R <= 16) LR_DOWN(1);
    else if (R <= 32) LR_DOWN(2);
    else if (R <= 64) LR_DOWN(4);
    else LR_DOWN(8);
#undef LR_DOWN
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // channels per block: 256 per step, as many steps as leave four blocks per
    // compute unit (each block adds up its tile's slices once)
    const int64_t cols = (N + 255) / 256;
    int64_t steps = cols * tiles / (4 * (int64_t)device_cu_count());
    steps = steps < 1 ? 1 : (steps > 8 ? 8 : steps);
    const int nblocks = (int)((cols + steps - 1) / steps);
    const dim3 ugrid((uint32_t)(tiles * nblocks));
#define LR_UP(KS) \
    lora_up_kernel<KS><<<ugrid, 256, 0, stream>>>(work, B, scale, pl, M, N, R, n, slices, nblocks, (int)steps, base, Y)
    if (R <= 16) LR_UP(1);
    else if (R <= 32) LR_UP(2);
    else if (R <= 64) LR_UP(4);
    else LR_UP(8);
#undef LR_UP
    return hipGetLastError();
}

}  // namespace svdq
