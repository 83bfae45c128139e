// api.hip -- the C-ABI entry points of libsvdq that run on the GPU, plus the
// status helpers.  Each device call validates its arguments and the current
// device before enqueuing anything ("Bringing Nunchaku 4-bit Diffusion
// Inference to Diffusers", section "Hardware support": the GPU is validated
// and a clear error is raised instead of producing incorrect outputs).
#include <atomic>
#include <cstring>
#include <mutex>

#include "svdq.h"
#include "svdq_internal.h"

namespace svdq {
namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_device_state[kMaxDevices];   // 0 unknown, 1 gfx950, 2 other

svdq_status current_device_ok()
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return SVDQ_ERR_UNSUPPORTED_DEVICE;
    }
    if (dev >= kMaxDevices) return SVDQ_ERR_UNSUPPORTED_DEVICE;
    int st = g_device_state[dev].load(std::memory_order_acquire);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
            (void)hipGetLastError();
            return SVDQ_ERR_UNSUPPORTED_DEVICE;
        }
        st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        g_device_state[dev].store(st, std::memory_order_release);
    }
    return st == 1 ? SVDQ_OK : SVDQ_ERR_UNSUPPORTED_DEVICE;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }      // int32 index arrays

svdq_status check_common(int M, int K, int rank, svdq_precision prec)
{
    if (prec != SVDQ_INT4 && prec != SVDQ_MXFP4) return SVDQ_ERR_INVALID_ARG;
    if (M < 0 || K < 0) return SVDQ_ERR_INVALID_ARG;
    if (rank != SVDQ_RANK) return SVDQ_ERR_UNSUPPORTED;
    const int g = group_size(prec);
    if (K < g || K % g != 0) return SVDQ_ERR_SHAPE;
    if (!elems_ok(M, K)) return SVDQ_ERR_SHAPE;
    return SVDQ_OK;
}

bool norm_ok(svdq_norm n) { return n == SVDQ_NORM_NONE || n == SVDQ_NORM_RMS || n == SVDQ_NORM_LAYER; }

// the weight and output matrices of a linear
svdq_status check_linear_sizes(int M, int N, int K)
{
    return elems_ok(N, K) && elems_ok(M, N) ? SVDQ_OK : SVDQ_ERR_SHAPE;
}

}  // namespace

int device_cu_count()
{
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return 256;
    }
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) {
            (void)hipGetLastError();
            n = 256;
        }
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace svdq

using namespace svdq;

extern "C" const char *svdq_status_string(svdq_status status)
{
    switch (status) {
    case SVDQ_OK: return "ok";
    case SVDQ_ERR_INVALID_ARG: return "invalid argument (NULL pointer, bad enum or negative size)";
    case SVDQ_ERR_SHAPE:
        return "unsupported shape (a size is not the multiple the call requires: K of the group size, N of 8, ...)";
    case SVDQ_ERR_MISALIGNED: return "device pointer not 16-byte aligned";
    case SVDQ_ERR_UNSUPPORTED:
        return "unsupported configuration (rank other than 32, or a precision or K the call does not support)";
    case SVDQ_ERR_UNSUPPORTED_DEVICE: return "no HIP device, or the current device is not a gfx950 (MI355X)";
    case SVDQ_ERR_NONFINITE: return "non-finite weight, calibration statistic or smoothing factor";
    case SVDQ_ERR_HIP: return "HIP runtime or kernel launch failure";
    case SVDQ_ERR_SCRATCH:
        return "the call needs more scratch memory than the library's static buffer holds (SVDQ_NOALLOC_SCRATCH_BYTES)";
    case SVDQ_STATUS_INT_RANGE_: break;    // not a status: it only sizes the enum
    }
    return "unknown status";
}

extern "C" int svdq_version(void) { return 200; }

extern "C" svdq_status svdq_check_device(void) { return current_device_ok(); }

extern "C" svdq_status svdq_quantize_act(const uint16_t *X, int M, int K, const float *smooth,
                                         const uint16_t *down, int rank, svdq_precision prec, uint8_t *xq,
                                         void *xscale, float *h, void *stream)
{
    svdq_status st = check_common(M, K, rank, prec);
    if (st != SVDQ_OK) return st;
    // buffers of zero size may be NULL (empty tensors have no storage)
    if (!smooth || !down || (M > 0 && (!X || !xq || !xscale || !h))) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(smooth) || !aligned16(down) || !aligned16(xq) || !aligned16(xscale) ||
        !aligned16(h))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0) return SVDQ_OK;
    hipError_t e = launch_quant_act(X, M, K, smooth, down, prec, xq, xscale, h, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" svdq_status svdq_w4a4_linear(const uint8_t *xq, const void *xscale, const float *h,
                                        const uint8_t *wq, const void *wscale, const uint16_t *up,
                                        const uint16_t *bias, int M, int N, int K, int rank,
                                        svdq_precision prec, svdq_epilogue epi, uint16_t *Y, void *stream)
{
    svdq_status st = check_common(M, K, rank, prec);
    if (st != SVDQ_OK) return st;
    if (N < 0) return SVDQ_ERR_INVALID_ARG;
    if (epi != SVDQ_EPI_NONE && epi != SVDQ_EPI_GELU_TANH) return SVDQ_ERR_INVALID_ARG;
    if (N % 8 != 0) return SVDQ_ERR_SHAPE;
    if (check_linear_sizes(M, N, K) != SVDQ_OK) return SVDQ_ERR_SHAPE;
    // buffers of zero size may be NULL (empty tensors have no storage)
    if ((M > 0 && (!xq || !xscale || !h)) || (N > 0 && (!wq || !wscale || !up)) ||
        (M > 0 && N > 0 && !Y))
        return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(xscale) || !aligned16(h) || !aligned16(wq) || !aligned16(wscale) ||
        !aligned16(up) || !aligned16(Y) || (bias && !aligned16(bias)))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    hipError_t e = launch_w4a4_linear(xq, xscale, h, wq, wscale, up, bias, M, N, K, prec, epi, Y,
                                      (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" size_t svdq_w4a4_linear_splitk_workspace_bytes(int M, int N, int K, svdq_precision prec)
{
    if (M <= 0 || N <= 0 || K <= 0 || (prec != SVDQ_INT4 && prec != SVDQ_MXFP4)) return 0;
    if (K % group_size(prec) != 0) return 0;
    if (!elems_ok(M, K) || check_linear_sizes(M, N, K) != SVDQ_OK) return 0;
    if (current_device_ok() != SVDQ_OK) return 0;       // the split depends on the device's CU count
    return splitk_work_bytes(M, N, K, prec);
}

extern "C" svdq_status svdq_w4a4_linear_splitk(const uint8_t *xq, const void *xscale, const float *h,
                                               const uint8_t *wq, const void *wscale, const uint16_t *up,
                                               const uint16_t *bias, int M, int N, int K, int rank,
                                               svdq_precision prec, svdq_epilogue epi, uint16_t *Y, void *work,
                                               size_t work_bytes, void *stream)
{
    svdq_status st = check_common(M, K, rank, prec);
    if (st != SVDQ_OK) return st;
    if (N < 0) return SVDQ_ERR_INVALID_ARG;
    if (epi != SVDQ_EPI_NONE && epi != SVDQ_EPI_GELU_TANH) return SVDQ_ERR_INVALID_ARG;
    if (N % 8 != 0) return SVDQ_ERR_SHAPE;
    if (check_linear_sizes(M, N, K) != SVDQ_OK) return SVDQ_ERR_SHAPE;
    if ((M > 0 && (!xq || !xscale || !h)) || (N > 0 && (!wq || !wscale || !up)) ||
        (M > 0 && N > 0 && !Y))
        return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(xscale) || !aligned16(h) || !aligned16(wq) || !aligned16(wscale) ||
        !aligned16(up) || !aligned16(Y) || (bias && !aligned16(bias)) || (work && !aligned16(work)))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    const size_t need = splitk_work_bytes(M, N, K, prec);
    if (need > 0 && (!work || work_bytes < need)) return SVDQ_ERR_INVALID_ARG;
    hipError_t e = launch_w4a4_linear_splitk(xq, xscale, h, wq, wscale, up, bias, M, N, K, prec, epi, Y,
                                             (float *)work, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" size_t svdq_requant_workspace_bytes(int M, int N, int rank, svdq_precision prec)
{
    (void)rank;
    (void)prec;
    if (M <= 0 || N <= 0) return 0;
    return requant_work_bytes(M, N);
}

extern "C" svdq_status svdq_w4a4_linear_requant(const uint8_t *xq, const void *xscale, const float *h,
                                                const uint8_t *wq, const void *wscale, const uint16_t *up,
                                                const uint16_t *bias, int M, int N, int K, int rank,
                                                svdq_precision prec, svdq_epilogue epi, const float *smooth2,
                                                const uint16_t *down2, uint8_t *xq2, void *xscale2, float *h2,
                                                void *work, size_t work_bytes, void *stream)
{
    svdq_status st = check_common(M, K, rank, prec);
    if (st != SVDQ_OK) return st;
    if (N < 0) return SVDQ_ERR_INVALID_ARG;
    if (epi != SVDQ_EPI_NONE && epi != SVDQ_EPI_GELU_TANH) return SVDQ_ERR_INVALID_ARG;
    if (N % 64 != 0) return SVDQ_ERR_SHAPE;
    if (check_linear_sizes(M, N, K) != SVDQ_OK) return SVDQ_ERR_SHAPE;
    if (!requant_supported(M, N, K, prec)) return SVDQ_ERR_UNSUPPORTED;
    // buffers of zero size may be NULL (empty tensors have no storage)
    if ((M > 0 && (!xq || !xscale || !h)) || (N > 0 && (!wq || !wscale || !up || !smooth2 || !down2)) ||
        (M > 0 && N > 0 && (!xq2 || !xscale2 || !h2 || !work)))
        return SVDQ_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && work_bytes < svdq_requant_workspace_bytes(M, N, rank, prec)) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(xscale) || !aligned16(h) || !aligned16(wq) || !aligned16(wscale) ||
        !aligned16(up) || (bias && !aligned16(bias)) || !aligned16(smooth2) || !aligned16(down2) ||
        !aligned16(xq2) || !aligned16(xscale2) || !aligned16(h2) || !aligned16(work))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    hipError_t e = launch_w4a4_linear_requant(xq, xscale, h, wq, wscale, up, bias, M, N, K, prec, epi, smooth2,
                                              down2, xq2, xscale2, h2, (float *)work, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" svdq_status svdq_w4a4_linear_qkv_norm_rope(const uint8_t *xq, const void *xscale, const float *h,
                                                      const uint8_t *wq, const void *wscale, const uint16_t *up,
                                                      const uint16_t *bias, int M, int N, int K, int rank,
                                                      svdq_precision prec, const uint16_t *norm_q,
                                                      const uint16_t *norm_k, float eps, const float *rope_cos,
                                                      const float *rope_sin, uint16_t *Y, void *stream)
{
    svdq_status st = check_common(M, K, rank, prec);
    if (st != SVDQ_OK) return st;
    if (N < 0) return SVDQ_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return SVDQ_ERR_INVALID_ARG;      // finite, non-negative
    if (N % 384 != 0) return SVDQ_ERR_SHAPE;
    if (check_linear_sizes(M, N, K) != SVDQ_OK) return SVDQ_ERR_SHAPE;
    if (!requant_supported(M, N, K, prec)) return SVDQ_ERR_UNSUPPORTED;      // MXFP4: the LDS-DMA kernel's range
    // buffers of zero size may be NULL (empty tensors have no storage)
    if ((M > 0 && (!xq || !xscale || !h || !rope_cos || !rope_sin)) ||
        (N > 0 && (!wq || !wscale || !up || !norm_q || !norm_k)) || (M > 0 && N > 0 && !Y))
        return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(xscale) || !aligned16(h) || !aligned16(wq) || !aligned16(wscale) ||
        !aligned16(up) || !aligned16(Y) || (bias && !aligned16(bias)) || !aligned16(norm_q) || !aligned16(norm_k) ||
        !aligned16(rope_cos) || !aligned16(rope_sin))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    hipError_t e = launch_w4a4_linear_qknorm(xq, xscale, h, wq, wscale, up, bias, M, N, K, prec, norm_q, norm_k, eps,
                                             rope_cos, rope_sin, Y, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" svdq_status svdq_awq_w4a16_linear(const uint16_t *X, const uint8_t *wq, const float *wscale,
                                             const uint16_t *bias, int M, int N, int K, uint16_t *Y,
                                             void *stream)
{
    if (M < 0 || N < 0 || K < 0) return SVDQ_ERR_INVALID_ARG;
    if (K < 256 || K % 256 != 0) return SVDQ_ERR_SHAPE;
    if (!elems_ok(M, K) || check_linear_sizes(M, N, K) != SVDQ_OK) return SVDQ_ERR_SHAPE;
    // buffers of zero size may be NULL (empty tensors have no storage)
    if ((M > 0 && !X) || (N > 0 && (!wq || !wscale)) || (M > 0 && N > 0 && !Y)) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(wq) || !aligned16(wscale) || (bias && !aligned16(bias)) || !aligned16(Y))
        return SVDQ_ERR_MISALIGNED;
    svdq_status st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    hipError_t e = launch_awq_linear(X, wq, wscale, bias, M, N, K, Y, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

static Nf4Levels nf4_levels_arg()
{
    Nf4Levels lv;
    std::memcpy(lv.c, nf4_codebook_cached(), sizeof(lv.c));
    return lv;
}

extern "C" svdq_status svdq_nf4_dequantize(const uint8_t *wq, const uint8_t *qabs, const float *chunk_scale, int N,
                                           int K, uint16_t *Wd, void *stream)
{
    if (N < 0 || K < 0) return SVDQ_ERR_INVALID_ARG;
    if (K < 64 || K % 64 != 0) return SVDQ_ERR_SHAPE;
    if (!elems_ok(N, K)) return SVDQ_ERR_SHAPE;
    if (N > 0 && (!wq || !qabs || !chunk_scale || !Wd)) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(wq) || !aligned16(qabs) || !aligned16(chunk_scale) || !aligned16(Wd)) return SVDQ_ERR_MISALIGNED;
    svdq_status st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (N == 0) return SVDQ_OK;
    hipError_t e = launch_nf4_dequant(wq, qabs, chunk_scale, N, K, nf4_levels_arg(), Wd, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" svdq_status svdq_nf4_w4a16_linear(const uint16_t *X, const uint8_t *wq, const uint8_t *qabs,
                                             const float *chunk_scale, const uint16_t *bias, int M, int N, int K,
                                             uint16_t *Y, void *stream)
{
    if (M < 0 || N < 0 || K < 0) return SVDQ_ERR_INVALID_ARG;
    if (K < 64 || K % 64 != 0 || N % 8 != 0) return SVDQ_ERR_SHAPE;
    if (!elems_ok(M, K) || check_linear_sizes(M, N, K) != SVDQ_OK) return SVDQ_ERR_SHAPE;
    // buffers of zero size may be NULL (empty tensors have no storage)
    if ((M > 0 && !X) || (N > 0 && (!wq || !qabs || !chunk_scale)) || (M > 0 && N > 0 && !Y))
        return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(wq) || !aligned16(qabs) || !aligned16(chunk_scale) || (bias && !aligned16(bias)) ||
        !aligned16(Y))
        return SVDQ_ERR_MISALIGNED;
    svdq_status st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    hipError_t e = launch_nf4_linear(X, wq, qabs, chunk_scale, bias, M, N, K, nf4_levels_arg(), Y, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" svdq_status svdq_residual_norm(const void *r, svdq_stream_type stype, const uint16_t *y, int M, int D,
                                          svdq_norm post, const uint16_t *post_w, const uint16_t *gate, float alpha,
                                          svdq_norm pre, const uint16_t *pre_w, const uint16_t *pre_b,
                                          const uint16_t *scale, const uint16_t *shift, const int32_t *mod_index,
                                          int mod_rows, int mod_stride, float eps, void *r_out, uint16_t *x,
                                          void *stream)
{
    if (stype != SVDQ_STREAM_BF16 && stype != SVDQ_STREAM_FP32) return SVDQ_ERR_INVALID_ARG;
    if (!norm_ok(post) || !norm_ok(pre)) return SVDQ_ERR_INVALID_ARG;
    if (M < 0 || D < 0) return SVDQ_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || eps > 3.0e38f || !(alpha >= -3.0e38f && alpha <= 3.0e38f)) return SVDQ_ERR_INVALID_ARG;
    if (D < 8 || D % 8 != 0 || D > 16384 || !elems_ok(M, D)) return SVDQ_ERR_SHAPE;
    // without a block output there is no update; without x nothing to normalize
    if (M > 0 && y == nullptr && (post != SVDQ_NORM_NONE || post_w || gate || r_out)) return SVDQ_ERR_INVALID_ARG;
    if (M > 0 && (!r || (y && !r_out) || (!y && !x) || (x && (x == r || x == r_out)))) return SVDQ_ERR_INVALID_ARG;
    if (gate || scale || shift) {
        if (mod_rows < 1) return SVDQ_ERR_INVALID_ARG;
        if (mod_stride < D || mod_stride % 8 != 0 || !elems_ok(mod_rows, mod_stride)) return SVDQ_ERR_SHAPE;
        if (!mod_index && M % mod_rows != 0) return SVDQ_ERR_SHAPE;
    }
    if (!aligned16(r) || !aligned16(y) || !aligned16(post_w) || !aligned16(gate) || !aligned16(pre_w) ||
        !aligned16(pre_b) || !aligned16(scale) || !aligned16(shift) || !aligned4(mod_index) || !aligned16(r_out) ||
        !aligned16(x))
        return SVDQ_ERR_MISALIGNED;
    svdq_status st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0) return SVDQ_OK;
    ResidualNormArgs a{};
    a.r = r, a.y = y, a.post_w = post_w, a.gate = gate, a.pre_w = pre_w, a.pre_b = pre_b, a.scale = scale;
    a.shift = shift, a.r_out = r_out, a.x = x, a.M = M, a.D = D, a.post = post, a.pre = pre;
    a.alpha = alpha, a.eps = eps, a.rows_per_mod = 1;
    if (gate || scale || shift) {
        a.mod_index = mod_index, a.mod_rows = mod_rows, a.mod_stride = mod_stride;
        if (!mod_index) a.rows_per_mod = M / mod_rows;
    }
    hipError_t e = launch_residual_norm(a, stype == SVDQ_STREAM_FP32, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

static svdq_status check_lora(int M, int n_adapters)
{
    if (M < 0) return SVDQ_ERR_INVALID_ARG;
    if (n_adapters < 1 || n_adapters > SVDQ_LORA_MAX_ADAPTERS) return SVDQ_ERR_UNSUPPORTED;
    return elems_ok(M, 1) ? SVDQ_OK : SVDQ_ERR_SHAPE;
}

static svdq_status check_lora_down(int M, int K, int rank, int n_adapters)
{
    svdq_status st = check_lora(M, n_adapters);
    if (st != SVDQ_OK) return st;
    if (K < 0) return SVDQ_ERR_INVALID_ARG;
    if (rank < 8 || rank > SVDQ_LORA_MAX_RANK || rank % 8 != 0) return SVDQ_ERR_UNSUPPORTED;
    if (K < 8 || K % 8 != 0 || !elems_ok(M, K) || !elems_ok(n_adapters * rank, K)) return SVDQ_ERR_SHAPE;
    return SVDQ_OK;
}

extern "C" size_t svdq_lora_plan_bytes(int M, int n_adapters)
{
    return check_lora(M, n_adapters) == SVDQ_OK && M > 0 ? lora_plan_size(M, n_adapters) : 0;
}

extern "C" size_t svdq_lora_workspace_bytes(int M, int K, int rank, int n_adapters)
{
    if (check_lora_down(M, K, rank, n_adapters) != SVDQ_OK || M == 0) return 0;
    if (current_device_ok() != SVDQ_OK) return 0;       // the slices depend on the device's CU count
    return lora_work_bytes(M, K, rank, n_adapters);
}

extern "C" svdq_status svdq_lora_plan(const int32_t *index, int M, int n_adapters, void *plan, size_t plan_bytes,
                                      void *stream)
{
    svdq_status st = check_lora(M, n_adapters);
    if (st != SVDQ_OK) return st;
    if (M > 0 && (!index || !plan || plan_bytes < lora_plan_size(M, n_adapters))) return SVDQ_ERR_INVALID_ARG;
    if (!aligned4(index) || !aligned16(plan)) return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0) return SVDQ_OK;
    return launch_lora_plan(index, M, n_adapters, plan, (hipStream_t)stream) == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" svdq_status svdq_lora_linear(const uint16_t *X, const uint16_t *A, const uint16_t *B, const float *scale,
                                        const void *plan, const uint16_t *base, int M, int N, int K, int rank,
                                        int n_adapters, uint16_t *Y, void *work, size_t work_bytes, void *stream)
{
    svdq_status st = check_lora_down(M, K, rank, n_adapters);
    if (st != SVDQ_OK) return st;
    if (N < 0) return SVDQ_ERR_INVALID_ARG;
    if (N % 8 != 0 || !elems_ok(M, N) || !elems_ok((int64_t)n_adapters * N, rank)) return SVDQ_ERR_SHAPE;
    if (M > 0 && N > 0 && (!X || !A || !B || !scale || !plan || !base || !Y || !work)) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(scale) || !aligned16(plan) ||
        !aligned16(base) || !aligned16(Y) || !aligned16(work))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    if (work_bytes < lora_work_bytes(M, K, rank, n_adapters)) return SVDQ_ERR_INVALID_ARG;
    hipError_t e = launch_lora_linear(X, A, B, scale, plan, base, M, N, K, rank, n_adapters, Y, (float *)work,
                                      (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

// Sizes of a cache, and the view of it that the kernels take.
static svdq_status check_kv4(const svdq_kv4_cache *c, Kv4View &v)
{
    if (!c || (c->prec != SVDQ_INT4 && c->prec != SVDQ_MXFP4)) return SVDQ_ERR_INVALID_ARG;
    if (c->pages < 1 || c->heads < 1) return SVDQ_ERR_INVALID_ARG;
    if (c->dim != 64 && c->dim != 128) return SVDQ_ERR_UNSUPPORTED;
    int shift = 4;
    while (shift < 8 && (1 << shift) != c->page_size) ++shift;
    if ((1 << shift) != c->page_size) return SVDQ_ERR_UNSUPPORTED;
    if (c->heads > 65535 || ((int64_t)c->pages << shift) > INT32_MAX) return SVDQ_ERR_SHAPE;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales))
        return SVDQ_ERR_MISALIGNED;
    v.k_codes = c->k_codes, v.v_codes = c->v_codes, v.k_scales = c->k_scales, v.v_scales = c->v_scales;
    v.pages = c->pages, v.page_shift = shift, v.heads = c->heads, v.dim = c->dim, v.int4 = c->prec == SVDQ_INT4;
    return SVDQ_OK;
}

static bool kv4_stride_ok(int64_t ld, int heads, int dim)
{
    return ld >= (int64_t)heads * dim && ld % 8 == 0 && ld < ((int64_t)1 << 40);
}

extern "C" svdq_status svdq_kv4_append(const svdq_kv4_cache *cache, const uint16_t *K, const uint16_t *V, int64_t ldk,
                                       int64_t ldv, const int32_t *slots, int T, void *stream)
{
    Kv4View c;
    svdq_status st = check_kv4(cache, c);
    if (st != SVDQ_OK) return st;
    if (T < 0) return SVDQ_ERR_INVALID_ARG;
    if (!elems_ok(T, (int64_t)c.heads * c.dim)) return SVDQ_ERR_SHAPE;
    if (!kv4_stride_ok(ldk, c.heads, c.dim) || !kv4_stride_ok(ldv, c.heads, c.dim)) return SVDQ_ERR_SHAPE;
    if (T > 0 && (!K || !V || !slots)) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(K) || !aligned16(V) || !aligned4(slots)) return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (T == 0) return SVDQ_OK;
    hipError_t e = launch_kv4_append(c, K, V, ldk, ldv, slots, T, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

extern "C" svdq_status svdq_kv4_read(const svdq_kv4_cache *cache, const int32_t *slots, int T, float *K, float *V,
                                     void *stream)
{
    Kv4View c;
    svdq_status st = check_kv4(cache, c);
    if (st != SVDQ_OK) return st;
    if (T < 0) return SVDQ_ERR_INVALID_ARG;
    if (!elems_ok(T, (int64_t)c.heads * c.dim)) return SVDQ_ERR_SHAPE;
    if (T > 0 && (!K || !V || !slots)) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(K) || !aligned16(V) || !aligned4(slots)) return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (T == 0) return SVDQ_OK;
    return launch_kv4_read(c, slots, T, K, V, (hipStream_t)stream) == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

static svdq_status check_kv4_attention(const Kv4View &c, int T, int B, int heads_q, int max_q, int max_kv)
{
    if (T < 0 || B < 0 || heads_q < 1 || max_q < 1 || max_kv < 1) return SVDQ_ERR_INVALID_ARG;
    if (heads_q % c.heads != 0 || !elems_ok(T, (int64_t)heads_q * c.dim)) return SVDQ_ERR_SHAPE;
    return (int64_t)B * c.heads < (1 << 24) ? SVDQ_OK : SVDQ_ERR_SHAPE;
}

extern "C" size_t svdq_kv4_attention_workspace_bytes(const svdq_kv4_cache *cache, int T, int B, int heads_q, int max_q,
                                                     int max_kv)
{
    Kv4View c;
    if (check_kv4(cache, c) != SVDQ_OK || check_kv4_attention(c, T, B, heads_q, max_q, max_kv) != SVDQ_OK) return 0;
    if (T == 0 || B == 0 || current_device_ok() != SVDQ_OK) return 0;
    return kv4_attention_work_bytes(T, B, heads_q, c.heads, c.dim, max_q, max_kv);
}

extern "C" svdq_status svdq_kv4_attention(const svdq_kv4_cache *cache, const uint16_t *Q, int64_t ldq,
                                          const int32_t *block_table, int table_width, const int32_t *q_start,
                                          const int32_t *kv_len, int B, int T, int heads_q, int max_q, int max_kv,
                                          float scale, int causal, int window, uint16_t *O, float *lse, void *work,
                                          size_t work_bytes, void *stream)
{
    Kv4View c;
    svdq_status st = check_kv4(cache, c);
    if (st != SVDQ_OK) return st;
    st = check_kv4_attention(c, T, B, heads_q, max_q, max_kv);
    if (st != SVDQ_OK) return st;
    if (!(scale > 0.0f) || scale > 2.0e38f || (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal))
        return SVDQ_ERR_INVALID_ARG;
    if (!kv4_stride_ok(ldq, heads_q, c.dim)) return SVDQ_ERR_SHAPE;
    if (table_width < 1) return SVDQ_ERR_INVALID_ARG;
    if (((int64_t)table_width << c.page_shift) > INT32_MAX - 4096) return SVDQ_ERR_SHAPE;
    if (T > 0 && B > 0 && (!Q || !block_table || !q_start || !kv_len || !O)) return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned4(block_table) || !aligned4(q_start) || !aligned4(kv_len) || !aligned16(O) ||
        !aligned16(lse) || !aligned16(work))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (T == 0 || B == 0) return SVDQ_OK;
    const size_t need = kv4_attention_work_bytes(T, B, heads_q, c.heads, c.dim, max_q, max_kv);
    if (need > 0 && (!work || work_bytes < need)) return SVDQ_ERR_INVALID_ARG;
    hipError_t e = launch_kv4_attention(c, Q, ldq, block_table, table_width, q_start, kv_len, B, T, heads_q, max_q,
                                        max_kv, scale, causal, window, O, lse, (float *)work, (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}

// ------------------------------------------------ allocation-free split K
//
// svdq_w4a4_linear_splitk_noalloc keeps the split-K slice sums in this
// file-scope device array instead of a caller workspace.  Each device holds
// its own copy at its own address; host code must use that address (from
// hipGetSymbolAddress), never the array's name.
static __device__ __align__(256) float scratch[SVDQ_NOALLOC_SCRATCH_BYTES / sizeof(float)];

namespace {

std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices];     // device address of `scratch`, per device (null until looked up)

// Device address of this device's `scratch`, looked up once per device with
// that device current; null if the lookup fails.
void *scratch_address(int dev)
{
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *ptr = nullptr;
        if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess) {
            (void)hipGetLastError();
            return nullptr;
        }
        g_scratch_ptr[dev] = ptr;
    }
    return g_scratch_ptr[dev];
}

}  // namespace

extern "C" svdq_status svdq_w4a4_linear_splitk_noalloc(const uint8_t *xq, const void *xscale, const float *h,
                                                       const uint8_t *wq, const void *wscale, const uint16_t *up,
                                                       const uint16_t *bias, int M, int N, int K, int rank,
                                                       svdq_precision prec, svdq_epilogue epi, uint16_t *Y,
                                                       void *stream)
{
    svdq_status st = check_common(M, K, rank, prec);
    if (st != SVDQ_OK) return st;
    if (N < 0) return SVDQ_ERR_INVALID_ARG;
    if (epi != SVDQ_EPI_NONE && epi != SVDQ_EPI_GELU_TANH) return SVDQ_ERR_INVALID_ARG;
    if (N % 8 != 0) return SVDQ_ERR_SHAPE;
    if (check_linear_sizes(M, N, K) != SVDQ_OK) return SVDQ_ERR_SHAPE;
    if ((M > 0 && (!xq || !xscale || !h)) || (N > 0 && (!wq || !wscale || !up)) || (M > 0 && N > 0 && !Y))
        return SVDQ_ERR_INVALID_ARG;
    if (!aligned16(xq) || !aligned16(xscale) || !aligned16(h) || !aligned16(wq) || !aligned16(wscale) ||
        !aligned16(up) || !aligned16(Y) || (bias && !aligned16(bias)))
        return SVDQ_ERR_MISALIGNED;
    st = current_device_ok();
    if (st != SVDQ_OK) return st;
    if (M == 0 || N == 0) return SVDQ_OK;
    const size_t need = splitk_work_bytes(M, N, K, prec);
    if (need > SVDQ_NOALLOC_SCRATCH_BYTES) return SVDQ_ERR_SCRATCH;
    float *work = nullptr;
    if (need > 0) {
        int dev = -1;
        if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
            (void)hipGetLastError();
            return SVDQ_ERR_HIP;
        }
        work = static_cast<float *>(scratch_address(dev));
        if (!work) return SVDQ_ERR_HIP;
    }
    // every slice of every tile is written in full before the finishing
    // kernel reads it, so the scratch needs no clearing
    hipError_t e = launch_w4a4_linear_splitk(xq, xscale, h, wq, wscale, up, bias, M, N, K, prec, epi, Y, work,
                                             (hipStream_t)stream);
    return e == hipSuccess ? SVDQ_OK : SVDQ_ERR_HIP;
}
