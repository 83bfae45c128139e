/*
 * svdq.h -- C ABI of libsvdq, an MI355X (gfx950) implementation of the
 * SVDQuant W4A4 linear layer.
 *
 * The layer ("Bringing Nunchaku 4-bit Diffusion Inference to Diffusers",
 * Hugging Face blog, section "Background: SVDQuant and Nunchaku"): a
 * per-channel smoothing moves activation outliers into the weights, the
 * hardest part of each smoothed weight matrix is kept in a small 16-bit
 * low-rank branch, and the residual runs as a 4-bit-weight x 4-bit-activation
 * product.  The low-rank down projection is fused with the activation
 * quantization, and the up projection with the 4-bit product (same section,
 * figure caption).  Section "Native loading in Diffusers" fixes rank 32 and a
 * bfloat16 compute dtype.
 *
 * Notation.  X is bf16 [M][K] (M tokens), W is bf16 [N][K] (nn.Linear
 * layout, out x in), y = X W^T + b.  r = rank = 32.  The 4-bit codes come in
 * groups along K: INT4 (symmetric, 64 wide, fp32 scale) or MXFP4 (E2M1
 * elements, one E8M0 scale per 32).
 *
 * Arithmetic (every step below is what the functions compute):
 *   s_k      = fl32(1 / sqrt(max|X_k| / max_n|W_nk|)), 1 when either max is 0
 *   What_kn  = W_nk / s_k ~ U S V^T (top r)
 *   down     = bf16(s_k (U S)_kj)   stored [r][K]  (K contiguous)
 *   up       = bf16(V_nj)           stored [N][r]  (r contiguous)
 *   residual R_kn = (W_nk - sum_j down[j][k] up[n][j]) / s_k, quantized from
 *            fl32(R) per (n, group)
 *   xhat     = fl32(X_mk s_k), quantized per (m, group);  h = X down^T (fp32)
 *   y        = sum_g sx_mg sw_ng (qx . qw)_g + h up^T + b   [GELU-tanh]  -> bf16
 * INT4 group: a = max|v|, scale = fl32(a / 7) (rounded upward instead of to
 * nearest below the normal fp32 range), code = round-half-even of the exact
 * quotient v / scale (always within [-7, 7]).  MXFP4 block: X = floor(log2 a)
 * - 2 clamped to [-127, 127], E8M0 = X + 127, element = v 2^-X rounded to the
 * E2M1 grid (ties to the even index, saturating at 6, sign kept for zero).
 * Codes are nibble-packed, element 2i in the low nibble of byte i.  Both code
 * formats are sign-magnitude with the sign of the input in bit 3 (kept for
 * zero): INT4 code = sign << 3 | |q|, E2M1 code = sign << 3 | grid index.
 *
 * Layout choices (the pages fix none of them):
 *   - down is stored [r][K] and up [N][r], i.e. both factors transposed
 *     against the textbook L1 [K][r], L2 [r][N]: the activation kernel reads
 *     16 consecutive channels of all 32 ranks as 32-byte runs, and the
 *     product's epilogue reads one output channel's 32 ranks as one 64-byte
 *     line.
 *   - INT4 codes are sign-magnitude, not two's complement: a sign-magnitude
 *     code becomes the exact fp8 (E4M3) byte of q 2^-9 with bit operations
 *     only, which is how the product feeds the matrix cores.
 *   - N % 8 == 0 for the linears: every row of Y, bias and up then starts on
 *     a 16-byte boundary.
 *
 * Conventions.
 *   - Ownership: the caller allocates and frees every buffer.  No call
 *     allocates device memory or keeps a pointer after it returns.
 *   - Device calls (svdq_quantize_act, svdq_w4a4_linear,
 *     svdq_w4a4_linear_few, svdq_w4a4_linear_gated,
 *     svdq_w4a4_linear_requant, svdq_w4a4_linear_splitk,
 *     svdq_w4a4_linear_qkv_norm_rope, svdq_awq_w4a16_linear,
 *     svdq_residual_norm, svdq_lora_*, svdq_rope_table, svdq_qk_norm_rope,
 *     svdq_kv4_*) take device
 *     pointers and a hipStream_t (as void*, NULL = the null stream); they
 *     validate everything first, enqueue kernels on `stream` and return
 *     without synchronizing.  On any error nothing has been enqueued or
 *     written.  The current HIP device must be a gfx950; otherwise
 *     SVDQ_ERR_UNSUPPORTED_DEVICE is returned and nothing runs.
 *   - Host calls (svdq_pack_weights, svdq_pack_residual,
 *     svdq_awq_pack_weights, svdq_rope_frequencies) take host pointers,
 *     run synchronously on the CPU and need no GPU.
 *   - Device pointers must be 16-byte aligned, int32 index arrays 4-byte
 *     aligned (SVDQ_ERR_MISALIGNED).  A buffer whose size is zero (M == 0 or
 *     N == 0) may be NULL.
 *   - Inputs are expected finite; the device calls do not check the values
 *     of X (non-finite X gives unspecified codes).
 *   - Every function is thread-safe.  Calls that overlap on one stream are
 *     ordered by the stream; calls on different streams that share output
 *     buffers race, as with any kernel.
 */
#ifndef SVDQ_H
#define SVDQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum svdq_status {
    SVDQ_OK = 0,
    SVDQ_ERR_INVALID_ARG = -1,        /* NULL pointer, bad enum value, negative size */
    SVDQ_ERR_SHAPE = -2,              /* a size not the multiple the call requires (K of the group, N of 8, ...),
                                         or a matrix of SVDQ_MAX_ELEMENTS elements or more */
    SVDQ_ERR_MISALIGNED = -3,         /* a device pointer not 16-byte aligned */
    SVDQ_ERR_UNSUPPORTED = -4,        /* rank other than 32, or a precision / K the call does not support */
    SVDQ_ERR_UNSUPPORTED_DEVICE = -5, /* no HIP device, or the current device is not gfx950 */
    SVDQ_ERR_NONFINITE = -6,          /* non-finite weight or calibration statistic (pack) */
    SVDQ_ERR_HIP = -7,                /* a HIP runtime or launch failure */
    SVDQ_ERR_SCRATCH = -8,            /* the allocation-free call needs more than SVDQ_NOALLOC_SCRATCH_BYTES */
    SVDQ_STATUS_INT_RANGE_ = 0x7FFFFFFF   /* not a status: makes every int a valid value of the type */
} svdq_status;

typedef enum svdq_precision {
    SVDQ_INT4 = 0,   /* symmetric INT4, 64-wide groups, fp32 scales  [rows][K/64] */
    SVDQ_MXFP4 = 1,  /* E2M1, 32-wide blocks, E8M0 scales (uint8)    [rows][K/32] */
    SVDQ_PRECISION_INT_RANGE_ = 0x7FFFFFFF   /* not a precision: every int is a valid value (calls reject it) */
} svdq_precision;

typedef enum svdq_epilogue {
    SVDQ_EPI_NONE = 0,
    SVDQ_EPI_GELU_TANH = 1, /* 0.5 y (1 + tanh(sqrt(2/pi) (y + 0.044715 y^3))) after the bias */
    SVDQ_EPILOGUE_INT_RANGE_ = 0x7FFFFFFF    /* not an epilogue: every int is a valid value (calls reject it) */
} svdq_epilogue;

/* Activation of a gated linear's gate. */
typedef enum svdq_activation {
    SVDQ_ACT_SILU = 0,       /* g / (1 + exp(-g)) */
    SVDQ_ACT_GELU_TANH = 1,  /* as SVDQ_EPI_GELU_TANH */
    SVDQ_ACTIVATION_INT_RANGE_ = 0x7FFFFFFF  /* not an activation: every int is a valid value (calls reject it) */
} svdq_activation;

typedef enum svdq_norm {
    SVDQ_NORM_NONE = 0,
    SVDQ_NORM_RMS = 1,      /* v / sqrt(mean(v^2) + eps) */
    SVDQ_NORM_LAYER = 2,    /* the same of v - mean(v) */
    SVDQ_NORM_INT_RANGE_ = 0x7FFFFFFF        /* not a norm: every int is a valid value (calls reject it) */
} svdq_norm;

typedef enum svdq_stream_type {
    SVDQ_STREAM_BF16 = 0,
    SVDQ_STREAM_FP32 = 1,
    SVDQ_STREAM_INT_RANGE_ = 0x7FFFFFFF      /* not a type: every int is a valid value (calls reject it) */
} svdq_stream_type;

/* Which channels of a head form the pairs that a rotation turns. */
typedef enum svdq_rope_pairs {
    SVDQ_ROPE_ADJACENT = 0,   /* pair p: channels 2 p and 2 p + 1 */
    SVDQ_ROPE_HALVES = 1,     /* pair p: channels p and pairs + p */
    SVDQ_ROPE_PAIRS_INT_RANGE_ = 0x7FFFFFFF  /* not a form: every int is a valid value (calls reject it) */
} svdq_rope_pairs;

/* How several axes share a head's pairs (sections[a] pairs of axis a, n in all). */
typedef enum svdq_rope_axes {
    SVDQ_ROPE_AXES_BLOCKS = 0,      /* runs of pairs, each with frequencies of its own: theta^(-j / sections[a]) */
    SVDQ_ROPE_AXES_SECTIONS = 1,    /* runs of pairs, the frequencies falling over all: theta^(-p / n) */
    SVDQ_ROPE_AXES_INTERLEAVED = 2, /* pair p: axis p % axes while p / axes is below that axis' number of pairs,
                                       else axis 0; theta^(-p / n) */
    SVDQ_ROPE_AXES_INT_RANGE_ = 0x7FFFFFFF   /* not a layout: every int is a valid value (calls reject it) */
} svdq_rope_axes;

#define SVDQ_RANK 32

/* Every matrix a call touches (M x K, N x K, M x N) must hold fewer than
 * this many elements (SVDQ_ERR_SHAPE otherwise), so that every byte offset
 * inside one buffer fits in 31 bits. */
#define SVDQ_MAX_ELEMENTS (1 << 30)

/* Human-readable text of a status code (static storage, never NULL). */
const char *svdq_status_string(svdq_status status);

/* Library version, major * 10000 + minor * 100 + patch. */
int svdq_version(void);

/* SVDQ_OK when the current HIP device is a gfx950, else
 * SVDQ_ERR_UNSUPPORTED_DEVICE.  Mirrors the capability check the pages
 * describe ("Hardware support": the quantizer validates the GPU at load time
 * and raises a clear error instead of producing incorrect outputs). */
svdq_status svdq_check_device(void);

/*
 * svdq_pack_weights -- host-side packing of one linear layer
 * ("Background: SVDQuant and Nunchaku": smoothing, low-rank branch,
 * 4-bit residual; "Native loading in Diffusers": rank 32).
 *
 *   W          [N][K] bf16 bits (nn.Linear weight, out x in), host
 *   act_absmax [K] fp32, per-channel max |X| from calibration (>= 0), host
 *   N, K       N >= 1; K >= group and K % group == 0 (group 64 INT4, 32 MXFP4)
 *   rank       must be 32
 *   prec       SVDQ_INT4 or SVDQ_MXFP4
 * Outputs (host, caller-allocated):
 *   smooth     [K] fp32                       s_k
 *   down       [rank][K] bf16 bits            bf16(s_k (U S)_kj)
 *   up         [N][rank] bf16 bits            bf16(V_nj)
 *   wq         [N][K/2] uint8                 packed residual codes
 *   wscale     INT4: [N][K/64] fp32; MXFP4: [N][K/32] uint8 (E8M0)
 * The top-r SVD is a randomized subspace iteration in fp64 with a
 * Rayleigh-Ritz step (not bit-reproducible against other SVD codes; signs:
 * the largest-|.| entry of each right singular vector is positive).  Columns
 * beyond the rank of the smoothed weight come out as zero.  Errors:
 * SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE, SVDQ_ERR_UNSUPPORTED, SVDQ_ERR_NONFINITE
 * (any non-finite W, or a negative / non-finite act_absmax).  Uses all host
 * cores (std::thread); outputs are deterministic.
 */
svdq_status svdq_pack_weights(const uint16_t *W, const float *act_absmax, int N, int K, int rank,
                              svdq_precision prec, float *smooth, uint16_t *down, uint16_t *up,
                              uint8_t *wq, void *wscale);

/*
 * svdq_pack_residual -- the residual step of svdq_pack_weights alone, for
 * caller-supplied smoothing and low-rank factors (same layouts as above):
 * R_kn = (W_nk - sum_j down[j][k] up[n][j]) / smooth_k in fp64, j ascending,
 * then fl32(R) quantized per (n, group).  Host, synchronous.  Errors as for
 * svdq_pack_weights (smooth must be finite and non-zero).
 */
svdq_status svdq_pack_residual(const uint16_t *W, const float *smooth, const uint16_t *down,
                               const uint16_t *up, int N, int K, int rank, svdq_precision prec,
                               uint8_t *wq, void *wscale);

/*
 * svdq_quantize_act -- fused activation step: smoothing, per-group absmax,
 * 4-bit quantization with nibble packing, and the rank-32 down projection
 * h = X down^T in the same pass over X ("Background: SVDQuant and Nunchaku":
 * the low-rank down projection is fused with the quantization kernel).
 *
 *   X        [M][K] bf16 bits, device          M >= 0 (M == 0: no-op)
 *   smooth   [K] fp32, device
 *   down     [rank][K] bf16 bits, device
 *   xq       [M][K/2] uint8, device (out)
 *   xscale   INT4: [M][K/64] fp32; MXFP4: [M][K/32] uint8, device (out)
 *   h        [M][rank] fp32, device (out)      fp32 accumulation of bf16 products
 *   stream   hipStream_t or NULL
 * Codes and scales are bit-exact with the definition above.  One kernel
 * launch.  Errors: SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE (K % group),
 * SVDQ_ERR_UNSUPPORTED (rank), SVDQ_ERR_MISALIGNED, SVDQ_ERR_UNSUPPORTED_DEVICE,
 * SVDQ_ERR_HIP.
 */
svdq_status svdq_quantize_act(const uint16_t *X, int M, int K, const float *smooth,
                              const uint16_t *down, int rank, svdq_precision prec, uint8_t *xq,
                              void *xscale, float *h, void *stream);

/*
 * svdq_w4a4_linear -- the 4-bit product with the fused low-rank up
 * projection, bias, optional GELU-tanh and bf16 store ("Background: SVDQuant
 * and Nunchaku": the up projection is fused with the 4-bit compute kernel;
 * "Introducing Nunchaku Lite": fused GELU/MLP paths).
 *
 *   xq, xscale, h   as written by svdq_quantize_act (device)
 *   wq, wscale      as written by svdq_pack_weights (device copies)
 *   up              [N][rank] bf16 bits (device)
 *   bias            [N] bf16 bits (device) or NULL
 *   M, N, K         M >= 0, N >= 0 (either 0: no-op), N % 8 == 0, K % group == 0
 *   epi             SVDQ_EPI_NONE or SVDQ_EPI_GELU_TANH
 *   Y               [M][N] bf16 bits (device, out), round-to-nearest-even
 * INT4: per 64-group exact integer partial products from the matrix
 * cores (each code enters the fp8 matrix instruction as an exact E4M3
 * value); the group scale sx * sw of each output comes from the bf16 matrix
 * instruction on high/low bf16 splits of both scales (relative error about
 * 2^-16) and multiplies the exact partial in one fp32 fma.  MXFP4: the
 * scaled f8f6f4 matrix instruction applies both E8M0 scales.  The low-rank
 * term uses h split into a bf16 high and low part and accumulates onto the
 * 4-bit term on the matrix cores; the bias enters there too, exactly, as
 * one more bf16 product (the bias row against a column of ones).  One kernel
 * launch;
 * for INT4, two when the tiles left after whole rounds of one block per CU
 * are few: those tiles are then computed in 64 x 64 pieces with K split
 * across a block's waves and the partial sums added in a fixed order (so
 * their outputs may differ in low bf16 places from what the one-launch form
 * gives for the same rows; results are deterministic for a given shape).
 * Errors as for svdq_quantize_act.
 */
svdq_status svdq_w4a4_linear(const uint8_t *xq, const void *xscale, const float *h,
                             const uint8_t *wq, const void *wscale, const uint16_t *up,
                             const uint16_t *bias, int M, int N, int K, int rank,
                             svdq_precision prec, svdq_epilogue epi, uint16_t *Y, void *stream);

/*
 * svdq_w4a4_linear_few -- svdq_w4a4_linear for the few rows of a decoding step
 * (single tokens, a tree of drafted tokens), where the tiles of svdq_w4a4_linear
 * would leave most of the chip idle: one pass over the weights per 64 rows of X,
 * 16 weight rows or a few times that per block.  Faster than svdq_w4a4_linear for
 * up to 64 rows (measured for K 1024 .. 11008, N 1024 .. 28672), and for more while
 * M N stays below about 1.5 million (INT4 of K about 1024: 1 million): 256 rows of
 * 6144 channels, 128 of 12288.  Arguments as for svdq_w4a4_linear, with
 *   M            0 .. SVDQ_FEW_MAX_ROWS (SVDQ_ERR_UNSUPPORTED above: more rows, a
 *                batch of many trees, go to svdq_w4a4_linear)
 * INT4: exact integer sums per group, scale product and accumulation in fp32.
 * Partial sums over K are added in a fixed order, so results are deterministic;
 * they may differ from svdq_w4a4_linear's in the last bf16 places.  One kernel
 * launch.  Errors as for svdq_w4a4_linear.
 */
#define SVDQ_FEW_MAX_ROWS 256
svdq_status svdq_w4a4_linear_few(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                                 const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int N, int K,
                                 int rank, svdq_precision prec, svdq_epilogue epi, uint16_t *Y, void *stream);

/*
 * svdq_w4a4_linear_gated -- the first half of a gated MLP in one kernel: gate
 * and up projection, activation and product,
 *   Y_mf = act(y_mf) * y_m,F+f,   y = svdq_w4a4_linear of 2 F channels
 * in fp32 from the sums to one rounding.
 *   wq, wscale, up, bias   of 2 F output channels, the gate's F first, then the
 *                up projection's: the packed tensors of the two weights on top of
 *                each other (packed together, or apart with the same smoothing)
 *   M, F, K      M >= 0, F >= 0 (either 0: no-op), F % 8 == 0, K % group == 0
 *   act          svdq_activation
 *   Y            [M][F] bf16 bits, device (out)
 * Any M: few rows (how many depends on F and K) run as in svdq_w4a4_linear_few, more in
 * the tiles of svdq_w4a4_linear.  One kernel launch.  Errors as for
 * svdq_w4a4_linear.
 */
svdq_status svdq_w4a4_linear_gated(const uint8_t *xq, const void *xscale, const float *h, const uint8_t *wq,
                                   const void *wscale, const uint16_t *up, const uint16_t *bias, int M, int F, int K,
                                   int rank, svdq_precision prec, svdq_activation act, uint16_t *Y, void *stream);

/*
 * svdq_w4a4_linear_splitk_workspace_bytes -- device workspace that
 * svdq_w4a4_linear_splitk needs on the current device: S * M * N fp32
 * partial sums when the MXFP4 product is split into S slices of K (S of 2
 * to 4; every slice but the last at least 1024 channels), else 0 (INT4,
 * shapes whose 256 x 256 tiles already fill half the chip, K < 2048 or
 * K % 256 != 0, M or N <= 0, invalid arguments, or no gfx950 device).
 * It depends on the device's compute-unit count.
 */
size_t svdq_w4a4_linear_splitk_workspace_bytes(int M, int N, int K, svdq_precision prec);

/*
 * svdq_w4a4_linear_splitk -- svdq_w4a4_linear for skinny shapes (few
 * tokens, long K, such as the MLP's second linear of a 512 x 512 image:
 * 1024 x 12288 -> 3072), where the product's tiles would leave most of the
 * chip idle.  Same arguments, arithmetic and output as svdq_w4a4_linear,
 * plus:
 *   work, work_bytes  device scratch of at least
 *                     svdq_w4a4_linear_splitk_workspace_bytes(M, N, K,
 *                     prec) bytes, 16-byte aligned (may be NULL when that
 *                     is 0); overwritten, caller-owned
 * With a split, each of S work items per tile sums its K slice into the
 * workspace in fp32, and a second kernel adds the S slices in slice order
 * (so the result is deterministic) before the epilogue; slice 0 adds the
 * low-rank term with the same bf16 high/low matrix product as the unsplit
 * epilogue, and the bias is added in fp32 after the slices.  Sums in a different
 * order than svdq_w4a4_linear's, so outputs may differ from it in the last
 * bf16 place.  Without a split it is svdq_w4a4_linear.  Errors as for
 * svdq_w4a4_linear, and SVDQ_ERR_INVALID_ARG for a NULL or too small work
 * (checked after the device, whose compute units set the size).
 */
svdq_status svdq_w4a4_linear_splitk(const uint8_t *xq, const void *xscale, const float *h,
                                    const uint8_t *wq, const void *wscale, const uint16_t *up,
                                    const uint16_t *bias, int M, int N, int K, int rank,
                                    svdq_precision prec, svdq_epilogue epi, uint16_t *Y, void *work,
                                    size_t work_bytes, void *stream);

/* Size of the library's static device scratch buffer (one per GPU, held
 * until the process ends), used by svdq_w4a4_linear_splitk_noalloc. */
#define SVDQ_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * svdq_w4a4_linear_splitk_noalloc -- svdq_w4a4_linear_splitk for callers
 * that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc): the same arguments,
 * kernels and results, without `work`: the split-K slice sums go to a
 * static device buffer of SVDQ_NOALLOC_SCRATCH_BYTES that the library holds
 * on each GPU it runs on.  The call itself allocates nothing (its first call
 * on a device looks up that device's buffer address once).
 *   - Shapes whose split needs more than SVDQ_NOALLOC_SCRATCH_BYTES
 *     (svdq_w4a4_linear_splitk_workspace_bytes) return SVDQ_ERR_SCRATCH and
 *     enqueue nothing.
 *   - Every call on one GPU shares that GPU's buffer: calls that overlap in
 *     time on one GPU (different streams, or different threads without
 *     ordering) race and give undefined results; calls on one stream are
 *     ordered and safe.  The buffer keeps the last call's contents; every
 *     call writes what it reads, so nothing needs clearing.
 * Errors as for svdq_w4a4_linear_splitk (without the workspace ones), plus
 * SVDQ_ERR_SCRATCH.
 */
svdq_status svdq_w4a4_linear_splitk_noalloc(const uint8_t *xq, const void *xscale, const float *h,
                                            const uint8_t *wq, const void *wscale, const uint16_t *up,
                                            const uint16_t *bias, int M, int N, int K, int rank,
                                            svdq_precision prec, svdq_epilogue epi, uint16_t *Y, void *stream);

/*
 * svdq_requant_workspace_bytes -- device workspace that
 * svdq_w4a4_linear_requant needs for M tokens and N output channels
 * (ceil(N / 256) * M * rank fp32 partial sums); 0 for M or N <= 0.
 */
size_t svdq_requant_workspace_bytes(int M, int N, int rank, svdq_precision prec);

/*
 * svdq_w4a4_linear_requant -- svdq_w4a4_linear feeding the next layer's
 * activation step directly (an MLP's fc1 -> fc2, "Introducing Nunchaku
 * Lite": fused GELU/MLP paths): Y is not stored.  Each output is rounded to
 * bf16 exactly as svdq_w4a4_linear would store it, then smoothed with the
 * next layer's `smooth2`, quantized per group of consecutive output channels
 * (64 INT4, 32 MXFP4), and multiplied into the next layer's `down2`.  The
 * results are those of svdq_quantize_act(Y, M, N, smooth2, down2, ...) on
 * that Y: codes and scales bit-exact, h2 up to the order of the fp32 sums
 * (per-tile partial sums over 256 channels, added in ascending tile order,
 * so h2 is deterministic).
 *
 *   xq ... epi   as for svdq_w4a4_linear; `prec` is that of both layers.
 *                MXFP4 needs K % 256 == 0 (SVDQ_ERR_UNSUPPORTED otherwise)
 *   N            N % 64 == 0 (the next layer's K)
 *   smooth2      [N] fp32, device                  next layer's s
 *   down2        [rank][N] bf16 bits, device       next layer's down
 *   xq2          [M][N/2] uint8, device (out)
 *   xscale2      INT4: [M][N/64] fp32; MXFP4: [M][N/32] uint8 (E8M0), device (out)
 *   h2           [M][rank] fp32, device (out)
 *   work         device scratch of at least svdq_requant_workspace_bytes(M,
 *                N, rank, prec) bytes, caller-owned; its contents on entry
 *                do not matter and are overwritten
 *   stream       hipStream_t or NULL
 * Two kernel launches on `stream` (the product with this epilogue, then the
 * fixed-order sum of the partial h2).  Errors: as for svdq_w4a4_linear;
 * SVDQ_ERR_SHAPE when N % 64 != 0; SVDQ_ERR_UNSUPPORTED for MXFP4 with
 * K % 256 != 0; SVDQ_ERR_INVALID_ARG when work_bytes is too small.
 */
svdq_status svdq_w4a4_linear_requant(const uint8_t *xq, const void *xscale, const float *h,
                                     const uint8_t *wq, const void *wscale, const uint16_t *up,
                                     const uint16_t *bias, int M, int N, int K, int rank,
                                     svdq_precision prec, svdq_epilogue epi, const float *smooth2,
                                     const uint16_t *down2, uint8_t *xq2, void *xscale2, float *h2,
                                     void *work, size_t work_bytes, void *stream);

/*
 * svdq_w4a4_linear_qkv_norm_rope -- svdq_w4a4_linear for a fused QKV
 * projection whose epilogue also applies the Q/K RMS-norm and the rotary
 * embedding ("Quantizing models with structural rewrites": the Nunchaku
 * engine's fused operator consumes the QKV projection, the Q/K normalization
 * and the rotary embeddings together).
 *
 *   xq ... bias  as for svdq_w4a4_linear; no GELU.  MXFP4 needs
 *                K % 256 == 0 (SVDQ_ERR_UNSUPPORTED otherwise)
 *   N            3 H 128 (SVDQ_ERR_SHAPE otherwise): channels [0, 128 H) are
 *                the Q heads, then H K heads, then H V heads, 128 each
 *   norm_q       [128] bf16 bits, device   RMS-norm weight of every Q head
 *   norm_k       [128] bf16 bits, device   RMS-norm weight of every K head
 *   eps          finite, >= 0 (SVDQ_ERR_INVALID_ARG otherwise)
 *   rope_cos     [M][64] fp32, device      cos of token m's angle for pair p
 *   rope_sin     [M][64] fp32, device      sin of the same angle
 *   Y            [M][N] bf16 bits, device (out)
 * With yb = the bf16 value svdq_w4a4_linear would store: V channels get yb;
 * a Q or K head gets u_d = yb_d / sqrt(mean_d(yb_d^2) + eps) * w_d (fp32),
 * then out_2p = u_2p cos_mp - u_2p+1 sin_mp, out_2p+1 = u_2p+1 cos_mp +
 * u_2p sin_mp, rounded to bf16 (round-to-nearest-even).  One kernel launch
 * (for INT4 two, with the leftover tiles in pieces, exactly when
 * svdq_w4a4_linear takes two at the same shape; yb is then that call's).
 * Errors as for svdq_w4a4_linear, plus the ones above.
 */
svdq_status svdq_w4a4_linear_qkv_norm_rope(const uint8_t *xq, const void *xscale, const float *h,
                                           const uint8_t *wq, const void *wscale, const uint16_t *up,
                                           const uint16_t *bias, int M, int N, int K, int rank,
                                           svdq_precision prec, const uint16_t *norm_q, const uint16_t *norm_k,
                                           float eps, const float *rope_cos, const float *rope_sin, uint16_t *Y,
                                           void *stream);

/*
 * svdq_awq_pack_weights -- host packing for the weight-only AWQ W4A16 layer
 * ("Native loading in Diffusers": the awq_w4a16 family, int4 with group size
 * 64, used for modulation layers, which are memory-bound and
 * precision-sensitive).  The activation-aware channel scaling of AWQ is a
 * calibration step; a caller that uses it passes the already scaled weight.
 *
 *   W        [N][K] bf16 bits, host            N >= 1, K >= 256, K % 256 == 0
 *   wq       [N][K/2] uint8, host (out)        codes q + 8, q in [-7, 7]
 *   wscale   [N][K/64] fp32, host (out)
 * q and the scale are the INT4 group quantizer of the header comment applied
 * to fl32(W) per (n, 64-group along k).  Storage order (the operand order of
 * the device kernel): in the 256-channel chunk C of a row, the 32 bytes at
 * 128 C + 32 b are 8 little-endian dwords d = 2 g + h; nibble j of dword d is
 * channel 256 C + 64 g + 32 h + 8 b + 2 j for j < 4 and + 2 (j - 4) + 1 for
 * j >= 4.  Host, synchronous, all host cores; errors SVDQ_ERR_INVALID_ARG,
 * SVDQ_ERR_SHAPE, SVDQ_ERR_NONFINITE (any non-finite W).
 */
svdq_status svdq_awq_pack_weights(const uint16_t *W, int N, int K, uint8_t *wq, float *wscale);

/*
 * svdq_awq_w4a16_linear -- y = X Wdq^T + b with Wdq_nk = wscale_ng q_nk and
 * bf16 activations (the awq_w4a16 runtime layer).
 *
 *   X        [M][K] bf16 bits, device          M >= 0 (0: no-op)
 *   wq, wscale   as written by svdq_awq_pack_weights (device copies)
 *   bias     [N] bf16 bits, device, or NULL
 *   N, K     N >= 0 (0: no-op), K >= 256, K % 256 == 0
 *   Y        [M][N] bf16 bits, device (out), round-to-nearest-even of the
 *            fp32 result
 *   stream   hipStream_t or NULL
 * Sums in fp32 on the bf16 matrix cores (each 64-channel group exactly, then
 * scaled once); the kernel streams the weights once per 16 rows of X, so it
 * is meant for the few rows of a modulation input.  One kernel launch.
 * Errors: SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE (K), SVDQ_ERR_MISALIGNED,
 * SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_awq_w4a16_linear(const uint16_t *X, const uint8_t *wq, const float *wscale,
                                  const uint16_t *bias, int M, int N, int K, uint16_t *Y, void *stream);

/*
 * NF4 weight-only W4A16 layer -- the pages' comparison system
 * ("BitsAndBytes W4 Quantization", sections "Overview" and "Parameters":
 * BF16 weights quantized at load time to the 4-bit "nf4" data type,
 * activations kept in bf16; compress_statistics double-quantizes the block
 * scaling statistics).
 *
 * Format.  Levels: 16 fp32 quantiles of the standard normal distribution
 * normalized to [-1, 1] with an exact zero (svdq_nf4_codebook).  A block is
 * 64 consecutive weights of a row, with absmax a (fp32); a weight's code is
 * the level nearest to fl32(w / a) (a tie goes to the level of smaller
 * magnitude; a == 0 gives the zero level, code 7).  The block absmaxes, in
 * row-major (n, block) order, are double-quantized in chunks of 256: s =
 * max a over the chunk, the chunk stores d = fl32(s / 255) and block b stores
 * q_b = round-half-even of 255 a_b / s.  Dequantized weight:
 *   ahat_b = fl32(q_b * d),   w' = bf16(fl32(level[code] * ahat_b)).
 */

/* The 16 NF4 levels, ascending (level 7 is 0, levels 0 and 15 are -1 and 1);
 * host, writes 16 floats.  Error: SVDQ_ERR_INVALID_ARG for NULL. */
svdq_status svdq_nf4_codebook(float *levels);

/*
 * svdq_nf4_pack_weights -- host packing of one weight for the NF4 layer.
 *   W            [N][K] bf16 bits, host            N >= 1, K >= 64, K % 64 == 0
 *   wq           [N][K/2] uint8, host (out)        codes; in each group of 8
 *                consecutive weights of a row, byte i holds weight i (low
 *                nibble) and weight i + 4 (high nibble)
 *   qabs         [N K / 64] uint8, host (out)      statistic codes, (n, block) order
 *   chunk_scale  [ceil(N K / 64 / 256)] fp32, host (out)   d of each chunk
 * Synchronous, all host cores.  Errors: SVDQ_ERR_INVALID_ARG,
 * SVDQ_ERR_SHAPE, SVDQ_ERR_NONFINITE (any non-finite W).
 */
svdq_status svdq_nf4_pack_weights(const uint16_t *W, int N, int K, uint8_t *wq, uint8_t *qabs,
                                  float *chunk_scale);

/*
 * svdq_nf4_dequantize -- the dequantized weights w' as bf16 [N][K] (device),
 * from device copies of svdq_nf4_pack_weights' outputs.  One kernel launch
 * on `stream`.  Errors: SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE (K),
 * SVDQ_ERR_MISALIGNED, SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_nf4_dequantize(const uint8_t *wq, const uint8_t *qabs, const float *chunk_scale, int N, int K,
                                uint16_t *Wd, void *stream);

/*
 * svdq_nf4_w4a16_linear -- y = X W'^T + b, W' dequantized inside the kernel
 * (the same w' as svdq_nf4_dequantize), sums in fp32 on the bf16 matrix
 * cores, rounded once to bf16 (round-to-nearest-even).
 *   X            [M][K] bf16 bits, device          M >= 0 (0: no-op)
 *   wq, qabs, chunk_scale   device copies of svdq_nf4_pack_weights' outputs
 *   bias         [N] bf16 bits, device, or NULL
 *   N, K         N >= 0 (0: no-op), N % 8 == 0; K >= 64, K % 64 == 0
 *   Y            [M][N] bf16 bits, device (out)
 * One kernel launch.  Errors: SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE,
 * SVDQ_ERR_MISALIGNED, SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_nf4_w4a16_linear(const uint16_t *X, const uint8_t *wq, const uint8_t *qabs,
                                  const float *chunk_scale, const uint16_t *bias, int M, int N, int K, uint16_t *Y,
                                  void *stream);

/*
 * svdq_residual_norm -- the step between two linears of a transformer block:
 * the gated residual update with the norms before and after it and the
 * modulation of the next block's input, whose shift, scale and gate vectors a
 * modulation layer (svdq_awq_w4a16_linear) computes.  Per row m:
 *   t  = post(y_m) * post_w
 *   r' = r_m + alpha * gate_b * t                            -> r_out
 *   x  = (pre(r') * pre_w + pre_b) * (1 + scale_b) + shift_b -> x
 * in fp32 from the loads to the stores (x is formed from the unrounded r';
 * r_out and x are rounded once, to nearest even).  The sums of squares are
 * fp32, so a row's values must stay below about 1e19 in magnitude.
 *
 *   r          [M][D], stype, device            the residual stream
 *   stype      SVDQ_STREAM_BF16 or SVDQ_STREAM_FP32: type of r and r_out
 *   y          [M][D] bf16 bits, device, or NULL: the block's output.  NULL:
 *              r' = r, and r_out, post_w and gate must be NULL too and post NONE
 *   M, D       M >= 0 (0: no-op); 8 <= D <= 16384, D % 8 == 0
 *   post, pre  norms; pre NONE and post NONE pass the values on
 *   post_w, pre_w, pre_b   [D] bf16 bits, device, or NULL (1, 1, 0)
 *   gate, scale, shift     row b at b * mod_stride, [mod_rows][D] bf16 bits
 *              (slices of one modulation output), device, or NULL (1, 0, 0)
 *   mod_index  [M] int32, device, or NULL: b of every row; a value outside
 *              [0, mod_rows) takes gate 1, scale 0, shift 0.  NULL: the rows
 *              are mod_rows equal runs (SVDQ_ERR_SHAPE unless M % mod_rows == 0)
 *   mod_rows, mod_stride   read when gate, scale or shift is given: mod_rows
 *              >= 1; mod_stride >= D, % 8 == 0; mod_rows * mod_stride below
 *              SVDQ_MAX_ELEMENTS
 *   alpha      residual scale, finite;   eps  finite, >= 0 (both norms)
 *   r_out      [M][D], stype, device (out); may be r itself
 *   x          [M][D] bf16 bits, device (out), or NULL: only r_out; pre and
 *              scale and shift are then not applied.  May be y itself, not r
 *              or r_out
 * One kernel launch.  Errors: SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE,
 * SVDQ_ERR_MISALIGNED, SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_residual_norm(const void *r, svdq_stream_type stype, const uint16_t *y, int M, int D,
                               svdq_norm post, const uint16_t *post_w, const uint16_t *gate, float alpha,
                               svdq_norm pre, const uint16_t *pre_w, const uint16_t *pre_b, const uint16_t *scale,
                               const uint16_t *shift, const int32_t *mod_index, int mod_rows, int mod_stride,
                               float eps, void *r_out, uint16_t *x, void *stream);

/*
 * Low-rank adapters of many requests beside a shared projection: every row
 * of a batch may carry its own adapter,
 *   Y_m = base_m + scale_a (X_m A_a^T) B_a^T,   a = index[m]
 * and rows without one keep base_m.  The batch's rows are grouped by adapter
 * once per step (svdq_lora_plan); the plan then serves every projection of
 * that step.
 */
#define SVDQ_LORA_MAX_RANK 128
#define SVDQ_LORA_MAX_ADAPTERS 4096

/* Device bytes of the plan of M rows and n_adapters adapters, and of the
 * workspace of svdq_lora_linear on the current device (it holds fp32 slices
 * of X A^T; their number depends on the device's compute units); 0 for sizes
 * the calls do not take, and without a gfx950 device for the workspace. */
size_t svdq_lora_plan_bytes(int M, int n_adapters);
size_t svdq_lora_workspace_bytes(int M, int K, int rank, int n_adapters);

/*
 * svdq_lora_plan -- groups M rows by adapter.
 *   index        [M] int32, device: adapter of every row; a value outside
 *                [0, n_adapters) means no adapter
 *   M            M >= 0 (0: no-op);  1 <= n_adapters <= SVDQ_LORA_MAX_ADAPTERS
 *   plan, plan_bytes   device, at least svdq_lora_plan_bytes(M, n_adapters)
 *                bytes, 16-byte aligned (out); valid until overwritten, read
 *                only by the calls that use it
 * One kernel launch (one block).  Errors: SVDQ_ERR_INVALID_ARG,
 * SVDQ_ERR_SHAPE (M), SVDQ_ERR_UNSUPPORTED (n_adapters),
 * SVDQ_ERR_MISALIGNED, SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_lora_plan(const int32_t *index, int M, int n_adapters, void *plan, size_t plan_bytes,
                           void *stream);

/*
 * svdq_lora_linear -- the adapters' part of a linear, added to `base`.
 *   X        [M][K] bf16 bits, device: the linear's input
 *   A        [n_adapters][rank][K] bf16 bits, device (down factors)
 *   B        [n_adapters][N][rank] bf16 bits, device (up factors)
 *   scale    [n_adapters] fp32, device
 *   plan     written by svdq_lora_plan for the same M and n_adapters (a plan
 *            of other sizes computes nothing)
 *   base     [M][N] bf16 bits, device: the shared projection's output
 *   M, N, K  M, N >= 0 (either 0: no-op); K >= 8; N % 8 == 0, K % 8 == 0
 *   rank     8 .. 128, rank % 8 == 0 (SVDQ_ERR_UNSUPPORTED otherwise);
 *            adapters of lower rank are padded with zero rows of A and zero
 *            columns of B
 *   Y        [M][N] bf16 bits, device (out); may be base itself (rows without
 *            an adapter are then not touched)
 *   work, work_bytes   device scratch of at least svdq_lora_workspace_bytes
 *            bytes, 16-byte aligned, overwritten (calls, or replays of captured
 *            ones, that may run at the same time need one each)
 * X A^T is summed in fp32 and enters the second product as a bf16 high and
 * low part (16 bits of significand); that product, the scale and the sum with
 * base are fp32, rounded once to bf16.  A row's result depends on that row
 * and the sizes alone, so it is deterministic.  The work is divided for the
 * most tiles that M and n_adapters allow, so A and B of the adapters in use
 * alone take less time than a large pool's.  Two kernel launches.  Errors:
 * SVDQ_ERR_INVALID_ARG (a too small workspace among them, checked after the
 * device), SVDQ_ERR_SHAPE, SVDQ_ERR_UNSUPPORTED, SVDQ_ERR_MISALIGNED,
 * SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_lora_linear(const uint16_t *X, const uint16_t *A, const uint16_t *B, const float *scale,
                             const void *plan, const uint16_t *base, int M, int N, int K, int rank, int n_adapters,
                             uint16_t *Y, void *work, size_t work_bytes, void *stream);

/*
 * Rotary positions with several axes (time, height and width of images and
 * video, or a single one).  Pair p of a head's channels turns by the angle
 *   angle_tp = pos[t][axis[p]] * freq[p]
 * whose cosine and sine a table holds, [T][pairs] fp32 each: the tables that
 * svdq_w4a4_linear_qkv_norm_rope takes (pairs = 64 there), made once per step
 * for all layers, or once for all positions with rows by position.
 */
#define SVDQ_ROPE_MAX_AXES 8

/*
 * svdq_rope_frequencies -- axis and frequency of every pair, on the host.
 *   sections   [axes] pairs of each axis, >= 0, their sum n <= 128, n % 8 == 0
 *   axes       1 .. SVDQ_ROPE_MAX_AXES;  theta  finite, > 0
 *   freq       [n] fp64 (out);  axis  [n] int32 (out)
 * Frequencies of another scheme (scaled for longer contexts, positions with a
 * unit of their own) are the caller's to write: the device calls take any.
 * Host, synchronous.  Errors: SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE (n).
 */
svdq_status svdq_rope_frequencies(const int *sections, int axes, double theta, svdq_rope_axes layout, double *freq,
                                  int32_t *axis);

/*
 * svdq_rope_table -- cosines and sines of T tokens' angles.
 *   pos        [T][axes] int32, device;  axes  1 .. SVDQ_ROPE_MAX_AXES
 *   freq       [pairs] fp64, device (radians per unit);  axis  [pairs] int32,
 *              device: a value outside [0, axes) does not turn (cos 1, sin 0)
 *   pairs      8 .. 128, pairs % 8 == 0
 *   cos, sin   [T][pairs] fp32, device (out)
 * The angle is the product rounded once to 64 bits; for angles below 2^30 the
 * results are within 2^-23 of its cosine and sine.  One kernel launch.  Errors:
 * SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE (pairs; T * pairs or T * axes of
 * SVDQ_MAX_ELEMENTS or more), SVDQ_ERR_MISALIGNED (pos and axis 4 bytes, freq 8,
 * cos and sin 16), SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_rope_table(const int32_t *pos, int T, int axes, const double *freq, const int32_t *axis, int pairs,
                            float *cos, float *sin, void *stream);

/*
 * svdq_qk_norm_rope -- RMS-norm and rotation of query and key heads:
 *   u = x / sqrt(mean_d(x_d^2) + eps) w (or x, without a weight);
 *   pair (a, b) of u -> (a cos - b sin, b cos + a sin); channels behind 2 pairs
 *   are u
 * rounded to bf16 (nearest even) once: queries from fp32, keys from 64 bits by way
 * of fp32, so that the 4 bits they may go on to are those of the exact key.
 *   Q, K       [T][heads_q][dim], [T][heads_k][dim] bf16 bits, device; row t
 *              at t * ldq, t * ldk elements (>= heads * dim, % 8 == 0): slices of
 *              a QKV product.  heads_q >= 1, heads_k >= 0 (0: K, K_out, norm_k are
 *              not read)
 *   dim        64, 128 or 256
 *   norm_q, norm_k   [dim] bf16 bits, device, or NULL: no norm on that side
 *   eps        finite, >= 0
 *   cos, sin   [table_rows][pairs] fp32, device;  pairs  8 .. dim / 2, % 8 == 0
 *   index      [T] int32, device: row of the tables for every token; a value
 *              outside [0, table_rows) does not turn (norm only).  NULL: row t of
 *              token t (tokens past table_rows do not turn)
 *   Q_out, K_out  as Q and K, rows at ldqo, ldko; may be Q and K themselves
 *              (with the same strides), not overlap them otherwise
 * One kernel launch.  Errors: SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE (strides,
 * pairs, T * heads * dim of SVDQ_MAX_ELEMENTS or more), SVDQ_ERR_UNSUPPORTED
 * (dim), SVDQ_ERR_MISALIGNED, SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_qk_norm_rope(const uint16_t *Q, int64_t ldq, int heads_q, const uint16_t *K, int64_t ldk,
                              int heads_k, int T, int dim, const uint16_t *norm_q, const uint16_t *norm_k, double eps,
                              const float *cos, const float *sin, const int32_t *index, int table_rows, int pairs,
                              svdq_rope_pairs style, uint16_t *Q_out, int64_t ldqo, uint16_t *K_out, int64_t ldko,
                              void *stream);

/*
 * 4-bit key / value cache: keys and values in the library's two 4-bit
 * formats, quantized along the head's channels by the same group quantizers
 * as activations and weights (header comment; INT4 64 wide, MXFP4 32 wide),
 * in pages that sequences share out through block tables.
 *
 * The caller allocates the four buffers, 16-byte aligned, of any content
 * (D = dim, g = 64 INT4 / 32 MXFP4, P = page_size):
 *   k_codes, v_codes     pages * heads * P * D / 2 bytes each
 *   k_scales, v_scales   pages * heads * P * D / g elements each, fp32 (INT4)
 *                        or uint8 E8M0 (MXFP4)
 * Layout, per page and head, tokens in runs of 16:
 *   k_codes [P/16][4][16][D/8] bytes: run, part b, token of the run, bytes.
 *           MXFP4: channel c in part c / (D/4), byte c % (D/4) / 2, nibble c %
 *           2; INT4: channel 64 g + 16 b + 8 s + i (b < 4, s < 2, i < 8) in
 *           part b, byte 8 g + 4 s + i % 4, nibble i / 4
 *   v_codes [P/16][4][16][D/32][4] bytes: run, token / 4, j, k, token % 4;
 *           channel 32 k + j in the low, 32 k + 16 + j in the high nibble
 *   k_scales, v_scales [P/16][D/g][16]: run, group, token
 * A token's slot is page * P + place.
 */
typedef struct svdq_kv4_cache {
    uint8_t *k_codes;
    void *k_scales;
    uint8_t *v_codes;
    void *v_scales;
    int pages;              /* >= 1; pages * page_size < 2^31 */
    int page_size;          /* 16, 32, 64, 128 or 256 tokens */
    int heads;              /* key / value heads, 1 .. 65535 */
    int dim;                /* channels per head: 64 or 128 */
    svdq_precision prec;
} svdq_kv4_cache;

/*
 * svdq_kv4_append -- quantizes T tokens' keys and values into their slots.
 *   K, V     [T][heads][dim] bf16 bits, device; row t at t * ldk, t * ldv
 *            elements (>= heads * dim, % 8 == 0): slices of a QKV product
 *   slots    [T] int32, device; a slot outside the cache skips that token.
 *            The slots of one call must differ (a slot given twice holds a
 *            mix of the two tokens afterwards)
 * Codes and scales are bit-exact with the definition in the header comment.
 * Values should be finite: a NaN is stored as some value of its group, an
 * infinity makes its group zeros (INT4) or is cut (MXFP4), so what a row does
 * not see cannot reach it.  Other slots keep their content.  One kernel launch.  Errors:
 * SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE (strides, cache sizes, T * heads * dim
 * of SVDQ_MAX_ELEMENTS or more), SVDQ_ERR_UNSUPPORTED (dim, page_size),
 * SVDQ_ERR_MISALIGNED, SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_kv4_append(const svdq_kv4_cache *cache, const uint16_t *K, const uint16_t *V, int64_t ldk,
                            int64_t ldv, const int32_t *slots, int T, void *stream);

/*
 * svdq_kv4_rope_append -- svdq_qk_norm_rope on the way into the cache: Q is
 * normed and rotated to Q_out, K is normed, rotated, rounded to bf16 and
 * appended with V as svdq_kv4_append does it (the codes are those of the two
 * calls).  Arguments as for these; heads and dim of K and V are the cache's.
 * One kernel launch.  Errors as for svdq_qk_norm_rope and svdq_kv4_append.
 */
svdq_status svdq_kv4_rope_append(const svdq_kv4_cache *cache, const uint16_t *Q, int64_t ldq, int heads_q,
                                 const uint16_t *K, const uint16_t *V, int64_t ldk, int64_t ldv,
                                 const uint16_t *norm_q, const uint16_t *norm_k, double eps, const float *cos,
                                 const float *sin, const int32_t *index, int table_rows, int pairs,
                                 svdq_rope_pairs style, const int32_t *slots, int T, uint16_t *Q_out, int64_t ldqo,
                                 void *stream);

/*
 * svdq_kv4_read -- the values that the cache holds for T slots:
 *   K, V     [T][heads][dim] fp32, device (out): fl32(code * scale); zeros for
 *            a slot outside the cache
 * One kernel launch.  Errors as for svdq_kv4_append.
 */
svdq_status svdq_kv4_read(const svdq_kv4_cache *cache, const int32_t *slots, int T, float *K, float *V,
                          void *stream);

/* Device bytes that are enough for svdq_kv4_attention and
 * svdq_kv4_tree_attention at these sizes on the current device (partial sums
 * where the keys are split over blocks); 0 without a split, for sizes they do
 * not take, or without a gfx950 device. */
size_t svdq_kv4_attention_workspace_bytes(const svdq_kv4_cache *cache, int T, int B, int heads_q, int max_q,
                                          int max_kv);

/*
 * svdq_kv4_attention -- attention of the last rows of B sequences over their
 * cached keys and values (the new tokens' own are appended first).
 *   Q            [T][heads_q][dim] bf16 bits, device; row t at t * ldq
 *                elements (>= heads_q * dim, % 8 == 0)
 *   block_table  [B][table_width] int32, device: the pages of each sequence in
 *                order.  Entries past a sequence's last page are not used; the
 *                keys of an entry outside [0, pages) are left out.  Pages that
 *                only hold keys that no row sees (behind a window) may be any,
 *                of any content
 *   q_start      [B + 1] int32, device, not decreasing: sequence s has the
 *                rows q_start[s] .. q_start[s + 1] - 1 (none: allowed).  Rows
 *                of no sequence keep what O and lse hold
 *   kv_len       [B] int32, device: keys of each sequence, the new tokens
 *                included; read up to table_width * page_size
 *   heads_q      a multiple of cache->heads: query head h uses key head
 *                h / (heads_q / heads)
 *   max_q, max_kv  >= 1, the caller's bounds on the rows and keys of a
 *                sequence.  They choose how the work is split, results for
 *                longer sequences are right as well
 *   scale        > 0, at most 2e38; multiplies the scores
 *   causal       0: a row sees all kv_len keys.  1: row i of n sees the keys
 *                up to place kv_len - n + i, itself included
 *   window       with causal: only the last `window` of these; 0: all
 *   O            [T][heads_q][dim] bf16 bits, device (out)
 *   lse          [T][heads_q] fp32, device (out), or NULL: log of the sum of
 *                exp(score)
 *   work, work_bytes  device scratch of at least
 *                svdq_kv4_attention_workspace_bytes bytes, 16-byte aligned,
 *                overwritten (NULL when that is 0; calls, or replays of
 *                captured ones, that may run at the same time need one each)
 * A row that sees no key gets zeros and lse -inf.  Scores, softmax and sums
 * are fp32 (a score must stay below 2e38 in magnitude, 256 times the sum of a
 * row's values of V within the range of fp32); the probabilities (INT4: times V's scale) enter the second
 * product rounded to bf16.  Deterministic for given sizes and bounds.  One
 * kernel launch, two with a split.  Errors: as for svdq_kv4_append, and
 * SVDQ_ERR_INVALID_ARG for a too small workspace (checked after the device).
 */
svdq_status svdq_kv4_attention(const svdq_kv4_cache *cache, const uint16_t *Q, int64_t ldq,
                               const int32_t *block_table, int table_width, const int32_t *q_start,
                               const int32_t *kv_len, int B, int T, int heads_q, int max_q, int max_kv, float scale,
                               int causal, int window, uint16_t *O, float *lse, void *work, size_t work_bytes,
                               void *stream);

/*
 * Drafted tokens as a tree.  The last rows of a sequence are tokens that a
 * draft proposes, each the child of another or of the sequence's last known
 * token: a step checks them all at once, a row seeing the known tokens, its
 * ancestors and itself.  kv_len counts the drafted tokens; they are appended at
 * their places in order (place kv_len - n + i of row i of n), however deep they
 * lie.
 */
#define SVDQ_TREE_MAX_WORDS 32      /* 1024 drafted tokens per sequence */

/*
 * svdq_kv4_tree_plan -- what the step needs of the tree, on the device.
 *   parent       [T] int32, device: the parent's number among its sequence's
 *                rows, smaller than the row's own; any other value: a child of
 *                the last known token
 *   q_start, kv_len, block_table, table_width, B, T   as for svdq_kv4_attention
 *   pages, page_size   of the cache
 *   mask         [T][mask_words] uint32, device (out): bit j % 32 of word j / 32
 *                is set where row j is the row itself or an ancestor; rows past
 *                32 mask_words are in no mask
 *   mask_words   1 .. SVDQ_TREE_MAX_WORDS
 *   position     [T] int32, device (out), or NULL: kv_len - n + the number of
 *                ancestors, the token's position in its text
 *   slots        [T] int32, device (out), or NULL: the slot of the row's place,
 *                -1 where the table has none and for rows of no sequence (a
 *                padded step's), so that appending writes nothing there
 * Rows of no sequence keep what mask and position hold.  One kernel launch.  Errors:
 * SVDQ_ERR_INVALID_ARG, SVDQ_ERR_SHAPE, SVDQ_ERR_UNSUPPORTED (page_size),
 * SVDQ_ERR_MISALIGNED (4 bytes), SVDQ_ERR_UNSUPPORTED_DEVICE, SVDQ_ERR_HIP.
 */
svdq_status svdq_kv4_tree_plan(const int32_t *parent, const int32_t *q_start, const int32_t *kv_len,
                               const int32_t *block_table, int table_width, int pages, int page_size, int B, int T,
                               uint32_t *mask, int mask_words, int32_t *position, int32_t *slots, void *stream);

/*
 * svdq_kv4_tree_attention -- svdq_kv4_attention of drafted tokens: row i of n
 * sees the keys before place kv_len - n, and the key at place kv_len - n + j
 * where bit j of its mask is set.
 *   mask, mask_words   as written by svdq_kv4_tree_plan, or any other: rows that
 *                see each other, or nothing (device, 4-byte aligned).  Bits past a
 *                sequence's rows are not used
 * All drafted tokens are appended first, those too that no row sees (what their
 * places hold has to be finite, as what svdq_kv4_append writes is).  There is no
 * window: every row sees all keys before the drafted ones.
 * Other arguments, workspace, arithmetic and errors as for svdq_kv4_attention.
 * Deterministic for given sizes, bounds and lengths: where the keys are split, how
 * they are cut, and so the last places of a row, may depend on the q_start and
 * kv_len of the whole batch.
 */
svdq_status svdq_kv4_tree_attention(const svdq_kv4_cache *cache, const uint16_t *Q, int64_t ldq,
                                    const int32_t *block_table, int table_width, const int32_t *q_start,
                                    const int32_t *kv_len, const uint32_t *mask, int mask_words, int B, int T,
                                    int heads_q, int max_q, int max_kv, float scale, uint16_t *O, float *lse,
                                    void *work, size_t work_bytes, void *stream);

/*
 * svdq_kv4_keep_path -- after the check: the accepted tokens' keys and values
 * close up behind the known ones, node path[i] to place kv_len - n + i.
 *   path         [B][max_path] int32, device: the accepted rows of every
 *                sequence, ascending from the first; it ends at the first that is
 *                negative, not above the one before it, or not below n
 *   max_path     >= 1
 *   new_len      [B] int32, device (out): kv_len - n + the path's length; not
 *                kv_len itself
 *   others       as for svdq_kv4_tree_plan
 * The bytes move as they are.  A place whose page is outside the cache is left
 * out of the move.  Places behind the path keep some of the drafted tokens.  One
 * kernel launch per layer's cache.  Errors: as for svdq_kv4_append.
 */
svdq_status svdq_kv4_keep_path(const svdq_kv4_cache *cache, const int32_t *path, int max_path,
                               const int32_t *q_start, const int32_t *kv_len, const int32_t *block_table,
                               int table_width, int B, int T, int32_t *new_len, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_H */
