// svdq_internal.h -- declarations shared between the C-ABI layer and the
// kernel translation units of libsvdq (not part of the public ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "svdq.h"

namespace svdq {

int group_size(svdq_precision prec);

// Every matrix a call touches (M x K, N x K, M x N) must hold fewer than
// SVDQ_MAX_ELEMENTS elements, so every byte offset inside one buffer fits in
// 31 bits: the LDS-DMA loads take 32-bit lane offsets and the host loops
// index rows with int products.
inline bool elems_ok(int64_t rows, int64_t cols) { return rows * cols < (int64_t)SVDQ_MAX_ELEMENTS; }

// Compute units of the current device (cached per device; 256 if unknown).
int device_cu_count();

// Kernel launchers; arguments are already validated.  They return the HIP
// status of the launch.
hipError_t launch_quant_act(const uint16_t *X, int M, int K, const float *smooth, const uint16_t *down,
                            svdq_precision prec, uint8_t *xq, void *xscale, float *h, hipStream_t stream);

hipError_t launch_w4a4_linear(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                              const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N,
                              int K, svdq_precision prec, svdq_epilogue epi, uint16_t *Y,
                              hipStream_t stream);

// Fused requantization: the product's epilogue writes the next layer's
// codes, scales and h instead of Y.  `work` holds the per-tile partial h
// (requant_work_bytes(M, N) bytes).  MXFP4 runs on the LDS-DMA kernel only
// (requant_supported).
size_t requant_work_bytes(int M, int N);
bool requant_supported(int M, int N, int K, svdq_precision prec);
hipError_t launch_w4a4_linear_requant(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                                      const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N,
                                      int K, svdq_precision prec, svdq_epilogue epi, const float *smooth2,
                                      const uint16_t *down2, uint8_t *xq2, void *xscale2, float *h2, float *work,
                                      hipStream_t stream);

// Split K for the MXFP4 linear when its 256 x 256 tiles fill less than half
// of the chip: S slices of K (S = 1: no split; `sps` steps of 256 channels
// per slice), fp32 partial sums in `work` (splitk_work_bytes, 0 without a
// split), then a fixed-order sum with the epilogue.  Without a split the
// launch is launch_w4a4_linear's.
int splitk_slices(int M, int N, int K, svdq_precision prec, int &sps);
size_t splitk_work_bytes(int M, int N, int K, svdq_precision prec);
hipError_t launch_w4a4_linear_splitk(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                                     const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N,
                                     int K, svdq_precision prec, svdq_epilogue epi, uint16_t *Y, float *work,
                                     hipStream_t stream);

// Linear of a QKV projection (N = 3 H 128) whose epilogue RMS-normalizes the
// Q and K heads and applies the rotary embedding.  MXFP4 runs on the LDS-DMA
// kernel only (requant_supported gives its range).
hipError_t launch_w4a4_linear_qknorm(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                                     const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N,
                                     int K, svdq_precision prec, const uint16_t *norm_q, const uint16_t *norm_k,
                                     float eps, const float *rope_cos, const float *rope_sin, uint16_t *Y,
                                     hipStream_t stream);

// Weight-only AWQ W4A16 layer (K % 256 == 0).
hipError_t launch_awq_linear(const uint16_t *X, const uint8_t *wq, const float *wscale, const uint16_t *bias,
                             int M, int N, int K, uint16_t *Y, hipStream_t stream);

// Weight-only NF4 W4A16 layer: the 16 fp32 levels (computed once on the
// host), the dequantization kernel and the linear.
struct Nf4Levels {
    float c[16];
};
const float *nf4_codebook_cached();
hipError_t launch_nf4_dequant(const uint8_t *wq, const uint8_t *qabs, const float *chunk, int N, int K,
                              const Nf4Levels &lv, uint16_t *Wd, hipStream_t stream);
hipError_t launch_nf4_linear(const uint16_t *X, const uint8_t *wq, const uint8_t *qabs, const float *chunk,
                             const uint16_t *bias, int M, int N, int K, const Nf4Levels &lv, uint16_t *Y,
                             hipStream_t stream);

// Gated residual, norms and modulation between two blocks (residual_norm.hip).
// y NULL: x from r alone; x NULL: the residual alone.
struct ResidualNormArgs {
    const void *r;
    const uint16_t *y, *post_w, *gate, *pre_w, *pre_b, *scale, *shift;
    const int32_t *mod_index;
    void *r_out;
    uint16_t *x;
    int M, D, post, pre, mod_rows, mod_stride, rows_per_mod;
    int grid_x;                     // blocks along x, set by the launch
    float alpha, eps;
};
hipError_t launch_residual_norm(const ResidualNormArgs &a, bool fp32, hipStream_t stream);

// Low-rank adapters of many requests (lora.hip).  The plan groups rows by
// adapter; `work` holds the slices of X A^T (lora_work_bytes).
constexpr int kLoraMaxRank = 128, kLoraMaxAdapters = 4096;
size_t lora_plan_size(int M, int n);
size_t lora_work_bytes(int M, int K, int R, int n);
hipError_t launch_lora_plan(const int32_t *index, int M, int n, void *plan, hipStream_t stream);
hipError_t launch_lora_linear(const uint16_t *X, const uint16_t *A, const uint16_t *B, const float *scale,
                              const void *plan, const uint16_t *base, int M, int N, int K, int R, int n, uint16_t *Y,
                              float *work, hipStream_t stream);

// 4-bit key / value cache (kv4.h has the layout; kv4_cache.hip,
// kv4_attention.hip).
struct Kv4View {
    uint8_t *k_codes, *v_codes;
    void *k_scales, *v_scales;
    int pages, page_shift, heads, dim;
    bool int4;
};
hipError_t launch_kv4_append(const Kv4View &c, const uint16_t *K, const uint16_t *V, int64_t ldk, int64_t ldv,
                             const int32_t *slots, int T, hipStream_t stream);
hipError_t launch_kv4_read(const Kv4View &c, const int32_t *slots, int T, float *K, float *V, hipStream_t stream);
// Splits of the keys keep their sums in `work` (0 bytes without a split).
size_t kv4_attention_work_bytes(int T, int B, int heads_q, int heads, int dim, int max_q, int max_kv);
hipError_t launch_kv4_attention(const Kv4View &c, const uint16_t *Q, int64_t ldq, const int32_t *table, int table_width,
                                const int32_t *q_start, const int32_t *kv_len, int B, int T, int heads_q, int max_q,
                                int max_kv, float scale, int causal, int window, uint16_t *O, float *lse, float *work,
                                hipStream_t stream);

}  // namespace svdq
