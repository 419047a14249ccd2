/*
 * fp8rl.h -- C ABI of libfp8rl, the GB300 (sm_103a) unified-precision FP8 linear layer.
 *
 * The scheme is the one stated in "Technical summary: Jet-RL" (gist.science, paper
 * 2601.14243), section "Quantization Scheme":
 *   - activations are quantized per 1x128 group,
 *   - weights are quantized per 128x128 block,
 *   - activations saved for the backward pass are stored in FP8 by the preceding (fused)
 *     operator, gradients passed between operators stay BF16,
 *   - DGrad and WGrad run in FP8, WGrad with 1x128 and 128x1 operand quantization.
 * Section "Core architecture" requires the inference (rollout) graph to be a sub-graph of
 * the training forward graph with the same quantization granularity and precision: the
 * same quantizers and GEMM numerics below serve both, including the small-M decode path.
 * Section "Implementation" names fused activation (SiLU-mul) and RMSNorm operators that
 * feed the quantizer; fp8rl_rmsnorm_quant and fp8rl_silu_mul_quant are those operators.
 *
 * Number formats and readings the pages leave open:
 *   - FP8 is OCP E4M3 ("FN": bias 7, max 448, no infinities).
 *   - A group's scale is s = fl32(amax / 448) in IEEE single precision; a group whose amax
 *     is 0 has s = 0 and all codes 0x00.
 *   - code = E4M3 round-to-nearest-even of fl32(x / s) (IEEE single division), saturated
 *     to +-448.  Dequantized value = decode(code) * s.
 *   - GEMMs multiply E4M3 codes exactly, accumulate each 128-long reduction block in FP32
 *     on the tensor cores, promote it into an FP32 accumulator with the product of the two
 *     operands' scales for that block, and round the result to BF16 (nearest even).
 *
 * Layouts (all row-major, element = one byte for codes, 4 bytes for scales, 2 bytes for
 * BF16 which travels as uint16_t bit patterns):
 *   1x128 codes of A[R,C]   : q[R][C]                 scales s[C/128][R]
 *   128x1 codes of X[M,K]   : emitted TRANSPOSED, qT[K][M]   scales sT[M/128][K]
 *                             (this is the 1x128 quantization of X^T along M)
 *   128x128 codes of W[N,K] : q[N][K]                 scales s[N/128][K/128]
 *                             optional transposed copy qT[K][N] uses the same scales.
 *
 * Shape rules: K % 128 == 0 always; N % 128 == 0 for weights and GEMM outputs; M % 128 == 0
 * wherever M is grouped 128x1 (the transposed outputs and WGrad).  M may be any value >= 0
 * elsewhere; M == 0 is a no-op that returns FP8RL_OK.  Other shapes return FP8RL_ERR_SHAPE.
 *
 * Memory and execution: the caller owns every buffer (device memory unless stated).  All
 * device pointers must be 16-byte aligned and every leading dimension a multiple of 16
 * bytes, else FP8RL_ERR_ALIGN.  Every call is asynchronous on the given stream; argument
 * errors are returned synchronously and launch nothing.  Device-side errors (a bounded
 * wait that ran out) are recorded in a per-device status word and returned by
 * fp8rl_check_status.  Inputs must be finite; NaN or Inf inputs give unspecified codes.
 * The library allocates no device memory of its own: split-K partial sums live in the
 * caller's workspace (fp8rl_gemm_workspace_bytes).
 *
 * Threading: the entry points are stateless apart from the status word and a per-device
 * cache of kernel attributes; they may be called from several host threads.  Each call
 * runs on the CUDA device that is current in the calling thread.
 */
#ifndef FP8RL_H
#define FP8RL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Exported from libfp8rl.so (the library is built with hidden visibility otherwise). */
#if defined(__GNUC__)
#define FP8RL_API __attribute__((visibility("default")))
#else
#define FP8RL_API
#endif

/* Same object as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* fp8rl_stream_t;

typedef enum {
    FP8RL_OK = 0,
    FP8RL_ERR_INVALID_ARG = 1,        /* null pointer, negative size, bad enum */
    FP8RL_ERR_SHAPE = 2,              /* a shape rule above is broken */
    FP8RL_ERR_ALIGN = 3,              /* pointer or leading dimension not 16-byte aligned */
    FP8RL_ERR_UNSUPPORTED_DEVICE = 4, /* current device is not compute capability 10.3 */
    FP8RL_ERR_WORKSPACE = 5,          /* workspace null or smaller than required */
    FP8RL_ERR_CUDA = 6,               /* a CUDA runtime/driver call failed */
    FP8RL_ERR_DEVICE_TIMEOUT = 7,     /* a kernel's bounded wait ran out (device status) */
    FP8RL_ERR_DEVICE_BOUNDS = 8       /* a kernel's own bounds check fired (device status) */
} fp8rl_status;

/* Library version, (major << 16) | minor. */
FP8RL_API int fp8rl_version(void);

/* Human-readable name of a status code (static string, never NULL). */
FP8RL_API const char* fp8rl_status_string(fp8rl_status st);

/* Checks that `device` is a compute-capability 10.3 GPU, makes it current in the calling
 * thread and prepares the kernels for it (function attributes).  Optional: every entry
 * point performs the same check for the current device on first use.  Returns
 * FP8RL_ERR_UNSUPPORTED_DEVICE on any other device, FP8RL_ERR_CUDA if CUDA fails. */
FP8RL_API fp8rl_status fp8rl_init(int device);

/* Upper bound, in nanoseconds, of every spin-wait inside the GEMM kernels (mbarrier waits
 * between the copy, tensor-core and epilogue warps).  When a wait runs out the kernel
 * records FP8RL_ERR_DEVICE_TIMEOUT, drains its own copies and returns.  Default 2e9 ns.
 * Applies to launches made after the call, on every device. */
FP8RL_API void fp8rl_set_wait_timeout_ns(uint64_t ns);

/* Waits for `stream`, then reads and clears the current device's status word.
 * Returns FP8RL_OK or the first device-side error recorded since the last check.
 * FP8RL_ERR_DEVICE_TIMEOUT means that the outputs of the GEMM calls made since the
 * previous check are not valid: a CTA whose wait ran out skips its stores (the split-K
 * reduction writes NaN instead once a timeout is on record). */
FP8RL_API fp8rl_status fp8rl_check_status(fp8rl_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * Quantizers ("Quantization Scheme": activations 1x128, weights 128x128, WGrad operands
 * 128x1; the transposed 128x1 output is the layout WGrad consumes).
 * -------------------------------------------------------------------------------------- */

/* Activation quantization, 1x128 groups along K.
 *   x  : BF16 [M][ldx] (first K columns used), ldx >= K
 *   q  : E4M3 [M][K];  s : float [K/128][M]
 *   qT, sT (both NULL or both set; then M % 128 == 0): the 128x1 quantization of the same
 *        x, transposed: qT [K][M], sT [M/128][K].  One read of x feeds both outputs. */
FP8RL_API fp8rl_status fp8rl_quantize_1x128(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                  uint8_t* q, float* s, uint8_t* qT, float* sT,
                                  fp8rl_stream_t stream);

/* 128x1 quantization along M (WGrad operand), transposed output.
 *   x : BF16 [M][ldx], M % 128 == 0;  qT : E4M3 [K][M];  sT : float [M/128][K] */
FP8RL_API fp8rl_status fp8rl_quantize_128x1(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                  uint8_t* qT, float* sT, fp8rl_stream_t stream);

/* 128x1 WGrad operand rebuilt from a saved 1x128 quantization (the memory-saving variant of
 * "Quantization Scheme": the activation saved for the backward pass is its FP8 form).
 *   q : E4M3 [M][K], s : float [K/128][M]  (an fp8rl_quantize_1x128 output)
 *   x^ = bf16_rne( fl32(decode(q) * s) ) is quantized 128x1 along M, transposed:
 *   qT : E4M3 [K][M], sT : float [M/128][K].  M % 128 == 0, K % 128 == 0.
 * The result differs from fp8rl_quantize_128x1 of the original BF16 X by the 1x128
 * rounding error it starts from. */
FP8RL_API fp8rl_status fp8rl_requantize_128x1(const uint8_t* q, const float* s, int64_t M, int64_t K,
                                              uint8_t* qT, float* sT, fp8rl_stream_t stream);

/* Weight quantization, 128x128 blocks (re-run from the BF16 master weights after each
 * optimizer step: "Core architecture", master weights stay BF16).
 *   w : BF16 [N][ldw];  q : E4M3 [N][K];  s : float [N/128][K/128]
 *   qT (nullable): E4M3 [K][N], the transposed copy DGrad reads; same scales. */
FP8RL_API fp8rl_status fp8rl_quantize_128x128(const uint16_t* w, int64_t N, int64_t K, int64_t ldw,
                                    uint8_t* q, float* s, uint8_t* qT,
                                    fp8rl_stream_t stream);

/* Fused RMSNorm -> quantize ("Implementation": fused RMSNorm kernel; "Quantization
 * Scheme": the saved activation is FP8, produced by the preceding operator).
 *   y[m,k] = bf16_rne( (x[m,k] * rstd[m]) * gamma[k] ),
 *   rstd[m] = 1 / sqrt( fl32(sum_k x[m,k]^2 / K) + eps )   (IEEE single sqrt and divide)
 * then y is quantized 1x128 (q [M][K], s [K/128][M]) and, if qT/sT are set, 128x1
 * transposed (qT [K][M], sT [M/128][K]; needs M % 128 == 0).  y itself is not stored.
 *   x : BF16 [M][K] (contiguous);  gamma : BF16 [K];  rstd (nullable): float [M] */
FP8RL_API fp8rl_status fp8rl_rmsnorm_quant(const uint16_t* x, const uint16_t* gamma, float eps,
                                 int64_t M, int64_t K, uint8_t* q, float* s, uint8_t* qT,
                                 float* sT, float* rstd, fp8rl_stream_t stream);

/* Fused SiLU-mul -> quantize ("Implementation": fused activation kernel).
 *   gu : BF16 [M][2*I], gate = columns [0, I), up = columns [I, 2I)
 *   h[m,i] = bf16_rne( silu(g) * u ), silu(g) = g / (1 + exp(-g)) evaluated in FP32
 * then h is quantized 1x128 (q [M][I], s [I/128][M]) and, if qT/sT are set, 128x1
 * transposed (qT [I][M], sT [M/128][I]).  I % 128 == 0. */
FP8RL_API fp8rl_status fp8rl_silu_mul_quant(const uint16_t* gu, int64_t M, int64_t I, uint8_t* q,
                                  float* s, uint8_t* qT, float* sT, fp8rl_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * Backward operators either side of the gradient quantizer ("Quantization Scheme":
 * gradients between operators stay BF16; DGrad and WGrad consume quantized gradients).
 * -------------------------------------------------------------------------------------- */

/* Fused SiLU-mul backward -> quantize: the gradient of the gate_up output from the forward's
 * gate_up output and the gradient of h (the down projection's DGrad output):
 *   gu : BF16 [M][2*I] (gate = columns [0, I), up = [I, 2I));  dh : BF16 [M][I]
 *   with s = sigmoid(g):  dg = bf16(dh*u*s*(1 + g*(1 - s))),  du = bf16(dh*g*s)
 *   evaluated in FP32; dgu = [dg | du] ([M][2I]) is quantized 1x128 along its 2I columns
 *   (q [M][2I], s [2I/128][M], the DGrad operand) and, if qT/sT are set (M % 128 == 0),
 *   128x1 transposed (qT [2I][M], sT [M/128][2I], the WGrad operand).  dgu itself is not
 *   stored.  I % 128 == 0. */
FP8RL_API fp8rl_status fp8rl_silu_mul_bwd_quant(const uint16_t* gu, const uint16_t* dh, int64_t M,
                                                int64_t I, uint8_t* q, float* s, uint8_t* qT,
                                                float* sT, fp8rl_stream_t stream);

/* RMSNorm backward from the forward's saved rstd (fp8rl_rmsnorm_quant's rstd output):
 *   x : BF16 [M][K];  gamma : BF16 [K];  rstd : float [M];  dy : BF16 [M][K] (the gradient
 *   of the normalised output)
 *   dx[m,j]   = bf16( r*gamma_j*dy_j - r^3*x_j*S/K ),  S = sum_k dy_k*gamma_k*x_k   (FP32)
 *   dgamma[k] = sum_m dy[m,k]*x[m,k]*r_m   (FP32; nullable: then ws is unused)
 * K % 128 == 0 and K <= 8192, else FP8RL_ERR_SHAPE.  dgamma needs
 * fp8rl_rmsnorm_bwd_workspace_bytes(M, K) bytes of workspace (no initial contents); the
 * sums run in a fixed order, so repeated calls give the same bits. */
FP8RL_API fp8rl_status fp8rl_rmsnorm_bwd(const uint16_t* x, const uint16_t* gamma, const float* rstd,
                                         const uint16_t* dy, int64_t M, int64_t K, uint16_t* dx,
                                         float* dgamma, void* ws, size_t ws_bytes,
                                         fp8rl_stream_t stream);
FP8RL_API size_t fp8rl_rmsnorm_bwd_workspace_bytes(int64_t M, int64_t K);

/* SiLU-mul -> quantize that also saves its input for the backward pass as an 8-bit
 * checkpoint, from one read of gu ("Quantization Scheme": activations saved for the backward
 * pass are FP8, produced by the fused operator).  q, s, qT, sT exactly as
 * fp8rl_silu_mul_quant; qgu (E4M3 [M][2I]), sgu (float [2I/128][M]) exactly as
 * fp8rl_quantize_1x128 of gu: half the bytes of gu, which need not be kept. */
FP8RL_API fp8rl_status fp8rl_silu_mul_quant_ckpt(const uint16_t* gu, int64_t M, int64_t I, uint8_t* q,
                                                 float* s, uint8_t* qT, float* sT, uint8_t* qgu,
                                                 float* sgu, fp8rl_stream_t stream);

/* fp8rl_silu_mul_bwd_quant from that checkpoint: the gate and up values are
 * decode(qgu) * sgu in FP32, everything else as there. */
FP8RL_API fp8rl_status fp8rl_silu_mul_bwd_quant_ckpt(const uint8_t* qgu, const float* sgu,
                                                     const uint16_t* dh, int64_t M, int64_t I,
                                                     uint8_t* q, float* s, uint8_t* qT, float* sT,
                                                     fp8rl_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * The norms before and after a block, fused with the block's gate, its residual scale, the
 * residual add and the quantizer of the next linear.  "Quantization Scheme": the activation
 * saved for the backward pass is FP8, produced by the preceding fused operator.
 *   n  = y r(y) g_post  (n = y when post_gamma is NULL),  r(v) = 1/sqrt(mean(v^2) + eps)
 *   h' = bf16_rne(h + alpha gate n)  (gate = 1 when NULL)
 *   z  = bf16_rne((h' r(h')) g_pre)
 * evaluated in FP32 (the squares too: a row whose sum of squares leaves FP32's range has r = 0,
 * as does one with an infinity; a NaN stays in its row; with eps = 0 a row of zeros has an infinite r).
 * The squares are added in FP32 without the error term that fp8rl_rmsnorm_quant's sum carries:
 * r is within 2^-20 of its value (a unit or two in the last place on ordinary rows, as
 * there), and the two operators' r of one row may differ in the last bits.  With post_gamma = gate = NULL and alpha = 1 this is the residual add
 * and norm of a pre-norm block.  A row's result depends on that row alone: a token gives
 * the same bits in a batch of one and in a training batch.
 * -------------------------------------------------------------------------------------- */
typedef struct {
    const uint16_t* h; int64_t ldh;    /* residual stream BF16 [M][ldh] */
    const uint16_t* y; int64_t ldy;    /* the block's output BF16 [M][ldy] */
    const uint16_t* post_gamma;        /* BF16 [K], nullable: no post norm */
    const uint16_t* gate;              /* BF16 [K], nullable */
    const uint16_t* pre_gamma;         /* BF16 [K] */
    float alpha, eps;                  /* residual scale; eps of both norms */
    uint16_t* h_out;                   /* h' BF16 [M][K]; may be h itself when ldh == K */
    uint16_t* z;                       /* BF16 [M][K], nullable */
    uint8_t* q; float* s;              /* z in 1x128: [M][K], [K/128][M]; both or neither */
    uint8_t* qT; float* sT;            /* z in 128x1, transposed: [K][M], [M/128][K]; both or
                                        * neither; needs M % 128 == 0 */
    uint8_t* qh; float* sh;            /* 8-bit checkpoint of h' (1x128); both or neither */
    uint8_t* qy; float* sy;            /* 8-bit checkpoint of y (1x128); both or neither */
    float* r_pre;                      /* r(h') [M] */
    float* r_post;                     /* r(y) [M]; needed with post_gamma */
} fp8rl_residual_norm_args;

/* At least one of z, q, qT is set.  K % 128 == 0 and K <= 8192, else FP8RL_ERR_SHAPE.  Other
 * than h_out on h, outputs overlap nothing. */
FP8RL_API fp8rl_status fp8rl_residual_norm(const fp8rl_residual_norm_args* args, int64_t M, int64_t K,
                                           fp8rl_stream_t stream);

/* Its gradients, from the gradients dz of z and dh of h' (dh NULL: zero) and the saved h', y,
 * r_pre, r_post.  h' and y are BF16, or both 8-bit checkpoints (qh/sh and qy/sy set: the
 * values decode(code) * scale, in FP32); y is read only with post_gamma or gate.
 *   x^ = h' r_pre,  t = dz g_pre,  dH = dh + r_pre (t - x^ mean(t x^))
 *   dn = alpha gate dH,  y^ = y r_post,  u = dn g_post,  dy = r_post (u - y^ mean(u y^))
 *   (dy = dn without a post norm)
 *   dpre = sum_m dz x^,  dpost = sum_m dn y^,  dgate = sum_m alpha dH n
 * dh_out = bf16(dH) is the gradient of h.  dpost is written with post_gamma, dgate with gate.
 * The sums run in a fixed order: repeated calls give the same bits.  The column sums are plain FP32
 * sums of M / 152 rows or fewer at a time (fp8rl_rmsnorm_bwd's carry an error term).  Every output overlaps
 * nothing.  ws: fp8rl_residual_norm_bwd_workspace_bytes(M, K), no initial contents. */
typedef struct {
    const uint16_t* dz; int64_t lddz;  /* BF16 [M][lddz] */
    const uint16_t* dh; int64_t lddh;  /* BF16 [M][lddh], nullable */
    const uint16_t* h; int64_t ldh;    /* h' BF16 [M][ldh], when qh is NULL */
    const uint8_t* qh; const float* sh;
    const uint16_t* y; int64_t ldy;    /* BF16 [M][ldy], when qy is NULL */
    const uint8_t* qy; const float* sy;
    const uint16_t* post_gamma;        /* BF16 [K], nullable */
    const uint16_t* gate;              /* BF16 [K], nullable */
    const uint16_t* pre_gamma;         /* BF16 [K] */
    float alpha;
    const float* r_pre;                /* [M] */
    const float* r_post;               /* [M], with post_gamma */
    uint16_t* dh_out;                  /* BF16 [M][K] */
    uint16_t* dy;                      /* BF16 [M][K] */
    float* dpre;                       /* [K] */
    float* dpost;                      /* [K], with post_gamma */
    float* dgate;                      /* [K], with gate */
} fp8rl_residual_norm_bwd_args;

FP8RL_API fp8rl_status fp8rl_residual_norm_bwd(const fp8rl_residual_norm_bwd_args* args, int64_t M, int64_t K,
                                               void* ws, size_t ws_bytes, fp8rl_stream_t stream);
FP8RL_API size_t fp8rl_residual_norm_bwd_workspace_bytes(int64_t M, int64_t K);

/* ----------------------------------------------------------------------------------------
 * Block-scaled FP8 GEMMs ("Quantization Scheme": forward, DGrad and WGrad in FP8).
 * Output element = bf16_rne( sum_kb sA(kb,row) * sB(kb,col) * sum_{k in kb} a*b ), with
 * the inner block sum in FP32 on the tensor cores and the outer sum in FP32 registers.
 * -------------------------------------------------------------------------------------- */

/* Operation selector for fp8rl_gemm_workspace_bytes and fp8rl_gemm_opts. */
typedef enum { FP8RL_OP_FWD = 0, FP8RL_OP_DGRAD = 1, FP8RL_OP_WGRAD = 2 } fp8rl_gemm_op;

/* Forward Y = X W^T.
 *   qx : E4M3 [M][K] (1x128), sx : float [K/128][M]
 *   qw : E4M3 [N][K] (128x128), sw : float [N/128][K/128]
 *   y  : BF16 [M][N]
 * Small M takes a decode-shaped form.  Up to 64 tokens (and up to 128 when N <= 8192),
 * FP8RL_VARIANT_DECODE: each CTA streams 128 weight rows of one reduction slice, and the
 * slices of a tile are added in rank order inside a cluster (the result does not depend
 * on timing); no workspace.  From 129 to 256 tokens against a weight wide enough that
 * the paired-SM form's 256-row tiles alone cover every pair of SMs, that form (below).
 * Otherwise up to 256 tokens, FP8RL_VARIANT_SPLITK: tokens on the tensor core's M side,
 * the reduction split over CTAs whose FP32 partial sums a second kernel adds in slice
 * order; it needs fp8rl_gemm_workspace_bytes(FP8RL_OP_FWD, M, N, K) bytes of workspace (no
 * initial contents required; calls that overlap in time need separate workspaces).  A
 * size of 0 means ws may be NULL.
 * Larger M takes the paired-SM form (FP8RL_VARIANT_PAIR, 256 x 256 tiles) when every
 * scale array can be moved by TMA -- M % 4 == 0 and (K/128) % 4 == 0 for the forward GEMM,
 * M % 4 == 0 and (K/128) % 4 == 0 on the weight's block-scale rows for DGrad -- and its
 * tiles cover every pair of SMs at least once; otherwise the one-SM tiled form
 * (FP8RL_VARIANT_TILED).  WGrad chooses the same way (its scale arrays always qualify). */
FP8RL_API fp8rl_status fp8rl_gemm_fwd(const uint8_t* qx, const float* sx, const uint8_t* qw,
                            const float* sw, uint16_t* y, int64_t M, int64_t N, int64_t K,
                            void* ws, size_t ws_bytes, fp8rl_stream_t stream);

/* DGrad dX = dY W.
 *   qdy : E4M3 [M][N] (1x128 along N), sdy : float [N/128][M]
 *   qwT : E4M3 [K][N], the transposed weight copy from fp8rl_quantize_128x128
 *   sw  : float [N/128][K/128] (the weight's block scales)
 *   dx  : BF16 [M][K]
 * ws may be NULL (no workspace is used at present). */
FP8RL_API fp8rl_status fp8rl_gemm_dgrad(const uint8_t* qdy, const float* sdy, const uint8_t* qwT,
                              const float* sw, uint16_t* dx, int64_t M, int64_t N,
                              int64_t K, void* ws, size_t ws_bytes, fp8rl_stream_t stream);

/* WGrad dW = dY^T X, both operands quantized 128x1 along the token dimension M.
 *   qdyT : E4M3 [N][M], sdyT : float [M/128][N]   (fp8rl_quantize_128x1 of dY)
 *   qxT  : E4M3 [K][M], sxT  : float [M/128][K]   (128x1 of the saved activation)
 *   dw   : BF16 [N][K];  M % 128 == 0. */
FP8RL_API fp8rl_status fp8rl_gemm_wgrad(const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT,
                              const float* sxT, uint16_t* dw, int64_t M, int64_t N,
                              int64_t K, void* ws, size_t ws_bytes, fp8rl_stream_t stream);

/* Workspace bytes the given GEMM needs with the automatic kernel choice (0 if none). */
FP8RL_API size_t fp8rl_gemm_workspace_bytes(int op, int64_t M, int64_t N, int64_t K);

/* Explicit kernel choice, for tests and benchmarks. */
typedef enum {
    FP8RL_VARIANT_AUTO = 0,   /* what fp8rl_gemm_fwd / _dgrad / _wgrad pick */
    FP8RL_VARIANT_TILED = 1,  /* one SM per output tile: persistent 128 x BN tiles */
    FP8RL_VARIANT_SPLITK = 2, /* decode-shaped: the reduction of each 128x256 output tile
                                 is split over `splits` CTAs (forward only, M <= 256) */
    FP8RL_VARIANT_PAIR = 3,   /* two SMs per output tile: persistent 256 x 256 (or, with
                                 tile_n = 128, 256 x 128) tiles on clusters of two CTAs
                                 (M = 256 tensor-core MMAs); needs
                                 scale arrays whose rows are multiples of 16 bytes (the
                                 rule under fp8rl_gemm_fwd), else FP8RL_ERR_SHAPE */
    FP8RL_VARIANT_DECODE = 4, /* forward only, M <= 256: weights on the MMA's M side (one
                                 CTA per 128 weight rows and reduction slice), the
                                 reduction split over a cluster of `splits` CTAs (1..8, 0 =
                                 choose) and summed in the cluster's shared memory in rank
                                 order; no workspace */
    FP8RL_VARIANT_MULTICAST = 5 /* the TILED form's 128 x 256 tiles on clusters of two CTAs
                                 (vertically adjacent tiles) that share each B tile: every
                                 CTA copies half of it with a TMA multicast into both CTAs;
                                 the same scale-array rule as PAIR (FP8RL_ERR_SHAPE
                                 otherwise); this GPU's memory only */
} fp8rl_variant;

typedef struct {
    int variant;    /* fp8rl_variant */
    int splits;     /* SPLITK: number of reduction slices (0 = choose); ignored otherwise */
    int grid;       /* TILED: persistent CTAs (0 = one per SM); PAIR, MULTICAST: persistent
                       clusters of two (0 = one per two SMs); ignored otherwise */
    int tile_n;     /* TILED: output tile width, 128 or 256 (0 = choose); PAIR: the pair
                       tile's width, 128 or 256 (0 = 256); ignored otherwise */
    int epi_warps;  /* PAIR: epilogue warps per CTA, 8 or 16 (0 = 8); ignored otherwise */
} fp8rl_gemm_opts;

/* Workspace bytes fp8rl_gemm_fwd_ex needs with these options (opts may be NULL = AUTO). */
FP8RL_API size_t fp8rl_gemm_workspace_bytes_ex(int op, int64_t M, int64_t N, int64_t K,
                                     const fp8rl_gemm_opts* opts);

/* fp8rl_gemm_fwd with an explicit variant; opts may be NULL (= AUTO). */
FP8RL_API fp8rl_status fp8rl_gemm_fwd_ex(const uint8_t* qx, const float* sx, const uint8_t* qw,
                               const float* sw, uint16_t* y, int64_t M, int64_t N,
                               int64_t K, void* ws, size_t ws_bytes,
                               const fp8rl_gemm_opts* opts, fp8rl_stream_t stream);

/* fp8rl_gemm_dgrad / fp8rl_gemm_wgrad with an explicit variant (AUTO, TILED, PAIR or
 * MULTICAST);
 * opts may be NULL (= AUTO). */
FP8RL_API fp8rl_status fp8rl_gemm_dgrad_ex(const uint8_t* qdy, const float* sdy, const uint8_t* qwT,
                                 const float* sw, uint16_t* dx, int64_t M, int64_t N,
                                 int64_t K, void* ws, size_t ws_bytes,
                                 const fp8rl_gemm_opts* opts, fp8rl_stream_t stream);
FP8RL_API fp8rl_status fp8rl_gemm_wgrad_ex(const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT,
                                 const float* sxT, uint16_t* dw, int64_t M, int64_t N,
                                 int64_t K, void* ws, size_t ws_bytes,
                                 const fp8rl_gemm_opts* opts, fp8rl_stream_t stream);

/* One linear layer from the BF16 activation ("Core architecture": rollout and the
 * training forward pass run the same FP8 linear): x is quantized 1x128 into qx / sx
 * (exactly fp8rl_quantize_1x128), then Y = X W^T with the form fp8rl_gemm_fwd picks.  In
 * the decode form without a cluster split, the GEMM kernel starts streaming its weights
 * while the quantizer finishes (programmatic dependent launch on the same stream).
 *   x : BF16 [M][ldx];  qw, sw, y, ws as for fp8rl_gemm_fwd;  qx : E4M3 [M][K] and
 *   sx : float [K/128][M] receive the quantized activation (caller-owned). */
FP8RL_API fp8rl_status fp8rl_linear_fwd(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                        const uint8_t* qw, const float* sw, int64_t N,
                                        uint8_t* qx, float* sx, uint16_t* y, void* ws,
                                        size_t ws_bytes, fp8rl_stream_t stream);

/* Decode-shaped forward GEMM that allocates nothing and takes no workspace.  It has no
 * counterpart in the scheme's pages; it exists for callers that cannot provide device
 * memory: a C/C++ decode loop that links only this library and owns no allocator, or a
 * serving loop that must not allocate between decode steps (allocating and freeing
 * device memory can synchronize the device and stall the loop).
 * Same operands, layouts and numerics as fp8rl_gemm_fwd_ex with FP8RL_VARIANT_SPLITK
 * and automatic splits (M <= 256); the result equals it within the GEMM tolerance (the
 * split, and with it the summation order, may differ).  Its split-K partial sums live in
 * a fixed scratch array inside the library,
 * fp8rl_gemm_noalloc_scratch_bytes() bytes (32 MiB) per device, reserved on every GPU
 * that loads the library and held until the process exits.
 *   - The automatic split keeps at most one (tile, slice) pair per SM, so the partial
 *     sums take at most SMs x 128 KiB (19 MiB on a 152-SM GB300); a GPU where they would
 *     not fit gets FP8RL_ERR_WORKSPACE.  M > 256 returns FP8RL_ERR_SHAPE.  Neither
 *     launches anything.
 *   - The first call in each CUDA context of a device looks up the array's device
 *     address (with that device current) and caches it; make that first call before any
 *     stream capture.
 *   - Every call on a device shares the array, which keeps the last call's partial sums
 *     (each call writes its own before reading them, so nothing needs clearing); calls
 *     whose kernels overlap on the GPU race on the array and give wrong results, so order
 *     them on one stream. */
FP8RL_API fp8rl_status fp8rl_gemm_fwd_decode_noalloc(const uint8_t* qx, const float* sx,
                                                     const uint8_t* qw, const float* sw,
                                                     uint16_t* y, int64_t M, int64_t N,
                                                     int64_t K, fp8rl_stream_t stream);

/* Size in bytes of the scratch array fp8rl_gemm_fwd_decode_noalloc uses on each device. */
FP8RL_API size_t fp8rl_gemm_noalloc_scratch_bytes(void);

/* ----------------------------------------------------------------------------------------
 * NVFP4 rollout path.  "QeRL" (chatpaper.ai), abstract: rollout runs with NVFP4-quantized
 * weights.  The page names the format only; the format is FP4 E2M1 elements (0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 and negatives), one E4M3 scale per 16 consecutive elements along K, and
 * an FP32 scale on top, here one per row.  The tensor core's FP4 path multiplies FP4 by
 * FP4, so the activation is quantized to NVFP4 as well, per call.
 *
 * Quantization of a row with maximum |x| = a (IEEE single precision, no FMA):
 *   g = a / 2688;  block of 16 with maximum b: sb = E4M3_rne_satfinite(b / (6 g)) (0 when
 *   g = 0), d = decode(sb) * g;  code = E2M1_rne_satfinite(x / d), 0 when d = 0.
 * Layouts:
 *   q  : [R][K/2] bytes; element k of a row in bits 4(k%2) .. 4(k%2)+3 of byte k/2.
 *   sf : the tensor core's scale-factor layout, fp8rl_nvfp4_scale_bytes(R, K) bytes:
 *        512-byte atoms of 128 rows x 4 scales (64 elements of K); atom (row group rg =
 *        r/128, K-atom ka = k/64) at byte 512 (rg K/64 + ka); inside it the scale of row
 *        r, K-elements 16j .. 16j+15 of the atom, at byte 16 (r%32) + 4 ((r%128)/32) + j.
 *        Rows from R up to the next multiple of 128 hold zeros.
 *   g  : float [R].
 * -------------------------------------------------------------------------------------- */

/* Bytes of the sf buffer of an R x K NVFP4 operand: ceil(R/128) * K/256 * 2048 (0 for
 * R <= 0 or K not a positive multiple of 256). */
FP8RL_API size_t fp8rl_nvfp4_scale_bytes(int64_t R, int64_t K);

/* NVFP4 quantization of the rows of x (BF16 [R][ldx], ldx >= K, ldx % 8 == 0; K % 256 == 0)
 * into q, sf, g (layouts above; caller-owned device memory, 16-byte aligned).  Used for
 * weights (R = N output channels, once per weight update) and activations (R = M tokens,
 * per call).  Errors: FP8RL_ERR_SHAPE (K % 256), FP8RL_ERR_ALIGN, FP8RL_ERR_INVALID_ARG. */
FP8RL_API fp8rl_status fp8rl_quantize_nvfp4(const uint16_t* x, int64_t R, int64_t K, int64_t ldx,
                                            uint8_t* q, uint8_t* sf, float* g, fp8rl_stream_t stream);

/* Decode-shaped NVFP4 GEMM: y[m][n] = bf16_rne(gx[m] gw[n] sum_k x^(m,k) w^(n,k)), x^ and
 * w^ the codes times their block scales, accumulated in FP32 by the tensor core (within
 * the GEMM tolerance of the exact sum).  Operands from fp8rl_quantize_nvfp4: qx / sfx / gx
 * of X [M][K], qw / sfw / gw of W [N][K].  y: BF16 [M][ldy], ldy >= N, ldy % 8 == 0.
 * 1 <= M <= 256, N % 128 == 0, K % 256 == 0.  splits: slices of the reduction, one cluster
 * of CTAs per 128-row weight tile (1..8; 0 = automatic).  No workspace. */
FP8RL_API fp8rl_status fp8rl_gemm_nvfp4(const uint8_t* qx, const uint8_t* sfx, const float* gx,
                                        const uint8_t* qw, const uint8_t* sfw, const float* gw,
                                        uint16_t* y, int64_t M, int64_t N, int64_t K, int64_t ldy,
                                        int splits, fp8rl_stream_t stream);

/* One NVFP4 linear layer from the BF16 activation: x is quantized into qx / sfx / gx
 * (exactly fp8rl_quantize_nvfp4; caller-owned), then y = fp8rl_gemm_nvfp4 with automatic
 * splits.  The GEMM kernel starts streaming its weights while the quantizer finishes
 * (programmatic dependent launch on the same stream) when the reduction is not split. */
FP8RL_API fp8rl_status fp8rl_linear_nvfp4(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                          const uint8_t* qw, const uint8_t* sfw, const float* gw,
                                          int64_t N, uint8_t* qx, uint8_t* sfx, float* gx,
                                          uint16_t* y, fp8rl_stream_t stream);

/* The same linear for 1 to 16 tokens with the activation left in BF16: only the weights are in
 * 4 bits.  y[m][n] = bf16_rne(gw[n] sum_k x[m][k] w^(n,k)), w^ the code times its block scale;
 * the products are exact (an element below 2^-28 of the largest of its 128 neighbours may lose
 * bits) and are summed in FP32 in a fixed order, in units of the fraction of gw[n] (its power of
 * two goes into the sum: a partial sum leaves FP32's range only where y's terms do).
 *   x : BF16 [M][ldx], ldx >= K, ldx % 8 == 0;  qw / sfw / gw as fp8rl_quantize_nvfp4 of W [N][K];
 *   y : BF16 [M][ldy], ldy >= N, ldy % 8 == 0.  0 <= M <= 16, N % 128 == 0, K % 256 == 0.
 * splits: CTAs of a cluster that share the reduction (1..8, or as many as K / 128 where that is
 * fewer; 0 = automatic).  A token's result
 * may differ in its last bit between calls of different M.  No workspace, one launch
 * (more only when K is so long that the tokens' x does not fit in shared memory at once).  A K
 * so long that one token's slice does not fit, above 45440 for each CTA that shares it, is
 * FP8RL_ERR_SHAPE for every M, before anything is launched.  y overlaps nothing. */
FP8RL_API fp8rl_status fp8rl_matvec_nvfp4(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                          const uint8_t* qw, const uint8_t* sfw, const float* gw,
                                          int64_t N, uint16_t* y, int64_t ldy, int splits,
                                          fp8rl_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * Expert layers: a router picks k of E experts for every token, the tokens' rows are brought
 * into expert order, every expert's rows are multiplied with its own weights by the scheme's
 * products, and the results are added up again per token.  The scheme's pages have dense layers
 * only; the quantization and numerics here are the same.
 *
 * Expert weights are one matrix W [E N][K], expert e's rows e N .. (e + 1) N, quantized by
 * fp8rl_quantize_128x128 as it stands: codes qw [E N][K], scales sw [E N / 128][K / 128] and the
 * transposed codes qwT [K][E N].
 *
 * A forward and backward of y = sum_j weight_j expert_j(x) reads:
 *   fp8rl_route_topk -> fp8rl_expert_rows -> fp8rl_expert_gather_quant(x) -> fp8rl_gemm_experts_fwd
 *   -> fp8rl_silu_mul_quant -> fp8rl_gemm_experts_fwd -> fp8rl_expert_combine(weight);
 *   fp8rl_expert_gather_quant(dout, weight) and fp8rl_expert_combine_dweight -> _dgrad, _wgrad ->
 *   fp8rl_silu_mul_bwd_quant -> _dgrad, _wgrad -> fp8rl_expert_combine(no weight) is dx;
 *   fp8rl_route_topk_bwd.
 * -------------------------------------------------------------------------------------- */

typedef enum { FP8RL_SCORE_SOFTMAX = 0, FP8RL_SCORE_SIGMOID = 1 } fp8rl_score;

typedef struct {
    const void* logits;   /* [T][ld], ld >= E: float, or BF16 with bf16 set */
    int64_t ld;
    int bf16;
    int score;            /* fp8rl_score */
    const float* bias;    /* [E], added to the scores for the selection only; NULL: none */
    int k;                /* experts of a token, 1 .. min(E, 32) */
    int n_groups;         /* equal groups of neighbouring experts (1 .. 32, divides E); 1: none */
    int top_groups;       /* groups that a token may choose from */
    int group_rank;       /* a group's rank is the sum of its 1 or 2 best */
    int renormalize;      /* weights divided by (their sum + 1e-20) */
    float scale;          /* multiplied into the weights */
    float* weight;        /* out [T][k] */
    int32_t* index;       /* out [T][k] */
} fp8rl_route_args;

/* The k experts of each token and their weights.  s = softmax or sigmoid of the logits,
 * v = s + bias (the logits themselves where there is neither a bias nor a group_rank of 2, which
 * gives the same order); among the experts of the top_groups best groups the k largest v, largest
 * first, the lowest index first among equals.  The order is that of the scores themselves, to
 * 2^-40, or 2^-44 of the largest |s + bias| where that is more: those too close for FP32 are formed
 * again in pairs of FP32.  weight = scale s / (sum of the k s + 1e-20), or scale s.
 *   An expert whose logit or bias is -inf is never chosen; where fewer than k can be, the rest of
 *   the row has index -1 and weight 0 (a padding token is a row of -inf).  NaN ranks above every
 *   number, so that it shows in the weights.
 * E <= 1024.  Pointers need the alignment of their elements only. */
FP8RL_API fp8rl_status fp8rl_route_topk(const fp8rl_route_args* args, int64_t T, int64_t E, fp8rl_stream_t stream);

typedef struct {
    const float* dweight;   /* [T][k] */
    const void* logits;     /* as in the forward */
    int64_t ld;
    int bf16;
    int score;
    const int32_t* index;   /* [T][k] the forward's; a value outside [0, E) is no expert */
    int k;
    int renormalize;
    float scale;
    void* dlogits;          /* out [T][ldd], ldd >= E, of the logits' type */
    int64_t ldd;
} fp8rl_route_bwd_args;

/* The gradient of the logits from that of the weights (the selection and the bias have none).
 * Experts given more than once in a row add up; masked logits get 0. */
FP8RL_API fp8rl_status fp8rl_route_topk_bwd(const fp8rl_route_bwd_args* args, int64_t T, int64_t E,
                                            fp8rl_stream_t stream);

/* Expert order of the T k pairs p = t k + j.  Expert e has the rows start[e] .. start[e] +
 * count[e], in the order of p; start[0] = 0 and start[e + 1] is the next multiple of `align` after
 * them.  Every buffer of rows has R = fp8rl_expert_rows_capacity(T, k, E, align) rows, the most
 * that the layout can need; rows that hold no pair are padding behind an expert or unused at the
 * end.  pos and src describe the same order, as fp8rl_expert_rows leaves them (a row whose pair is
 * not at that row in pos is not written by the gather).
 *   align = 128: training and prefill (the 128x1 groups and the GEMM tiles of an expert are its own);
 *   align = 1:   rollout, a few rows an expert (forward only; R = T k). */
typedef struct {
    const int32_t* pos;     /* [T][k] row of each pair, -1 for a pair of no expert */
    const int32_t* src;     /* [R] pair of each row, or -1 */
    const int32_t* start;   /* [E + 1] */
    const int32_t* count;   /* [E] */
    int64_t T, k, E, R, align;
} fp8rl_expert_layout;

/* R of a layout: the multiple of align at or below T k + min(E, T k) (align - 1); 0 where an
 * argument is out of its range. */
FP8RL_API int64_t fp8rl_expert_rows_capacity(int64_t T, int64_t k, int64_t E, int64_t align);

/* Sorts the pairs by expert: index [T][k] -> pos, src, start, count (all written; 4-byte aligned, as
 * in every call that takes them).  An index outside [0, E) is a pair of no expert; the same expert twice in a row
 * is two pairs.  1 <= k <= 32, E <= 1024, T k <= 2^30, align 1 or 128.  The workspace, of
 * fp8rl_expert_rows_workspace_bytes (0 for small calls), is written before it is read. */
FP8RL_API fp8rl_status fp8rl_expert_rows(const int32_t* index, int64_t T, int64_t k, int64_t E, int64_t align,
                                         int32_t* pos, int32_t* src, int32_t* start, int32_t* count, void* ws,
                                         size_t ws_bytes, fp8rl_stream_t stream);
FP8RL_API size_t fp8rl_expert_rows_workspace_bytes(int64_t T, int64_t k, int64_t E);

/* Row src[r] / k of x for every row r, quantized as fp8rl_quantize_1x128 does.
 *   x      : BF16 [T][ldx];  weight: float [T][k] or NULL: row r is bf16(weight[src[r]] x) then;
 *   q, s   : E4M3 [R][K], float [K/128][R];
 *   qT, sT : both NULL, or (align 128) the 128x1 quantization [K][R], [R/128][K].
 * Every row is written: those of no pair have codes and scales 0. */
FP8RL_API fp8rl_status fp8rl_expert_gather_quant(const uint16_t* x, int64_t ldx, int64_t K, const float* weight,
                                                 const fp8rl_expert_layout* rows, uint8_t* q, float* s, uint8_t* qT,
                                                 float* sT, fp8rl_stream_t stream);

/* out[t] = residual[t] + sum_j weight[t][j] y[pos[t][j]], summed in FP32 in the order of j; weight
 * NULL: 1; residual NULL: 0; pairs without a row add nothing.  With weight NULL it is the backward
 * of the gather.
 *   y : BF16 [R][ldy], residual [T][ldr], out [T][ldo], N columns, N % 8 == 0,
 *   at most 2^24.  out may be residual. */
FP8RL_API fp8rl_status fp8rl_expert_combine(const uint16_t* y, int64_t ldy, int64_t N, const float* weight,
                                            const uint16_t* residual, int64_t ldr, const fp8rl_expert_layout* rows,
                                            uint16_t* out, int64_t ldo, fp8rl_stream_t stream);

/* dweight[t][j] = <dout[t], y[pos[t][j]]> in FP32, 0 for a pair without a row.  (The gradient of y
 * is fp8rl_expert_gather_quant of dout with the weights.) */
FP8RL_API fp8rl_status fp8rl_expert_combine_dweight(const uint16_t* dout, int64_t ldd, const uint16_t* y, int64_t ldy,
                                                    int64_t N, const fp8rl_expert_layout* rows, float* dweight,
                                                    fp8rl_stream_t stream);

/* Y[r] = X[r] W_e^T for the rows r of each expert e.  qx, sx as fp8rl_expert_gather_quant gives them;
 * qw [E N][K], sw [E N / 128][K / 128]; y BF16 [R][N].  Rows behind the last expert's are left as
 * they were, padding rows get the product of their codes.
 *   align 128: 256 x 256 tiles on pairs of SMs;  align 1: a tile of 128 weight rows and up to 32
 *   or 64 token rows, for up to some tens of rows an expert (it is right for any number). */
FP8RL_API fp8rl_status fp8rl_gemm_experts_fwd(const uint8_t* qx, const float* sx, const uint8_t* qw, const float* sw,
                                              uint16_t* y, int64_t N, int64_t K, const fp8rl_expert_layout* rows,
                                              fp8rl_stream_t stream);

/* dX[r] = dY[r] W_e.  qdy [R][N], sdy [N/128][R]; qwT [K][E N]; sw as above; dx BF16 [R][K].
 * align 128. */
FP8RL_API fp8rl_status fp8rl_gemm_experts_dgrad(const uint8_t* qdy, const float* sdy, const uint8_t* qwT, const float* sw,
                                                uint16_t* dx, int64_t N, int64_t K, const fp8rl_expert_layout* rows,
                                                fp8rl_stream_t stream);

/* dW_e = sum over the rows r of expert e of dY[r]^T X[r], zeros for an expert without rows.
 * qdyT [N][R], sdyT [R/128][N], qxT [K][R], sxT [R/128][K]; dw BF16 [E N][K].  align 128. */
FP8RL_API fp8rl_status fp8rl_gemm_experts_wgrad(const uint8_t* qdyT, const float* sdyT, const uint8_t* qxT,
                                                const float* sxT, uint16_t* dw, int64_t N, int64_t K,
                                                const fp8rl_expert_layout* rows, fp8rl_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * Diagnostics (used by the tests).
 * -------------------------------------------------------------------------------------- */

/* The device's E4M3 encoder (the exact routine the quantizers use) applied to n binary32
 * values: out[i] = E4M3_rne_satfinite(in[i]).  Device pointers. */
FP8RL_API fp8rl_status fp8rl_debug_e4m3_encode(const float* in, uint8_t* out, int64_t n,
                                     fp8rl_stream_t stream);

/* The device's E2M1 encoder (the routine fp8rl_quantize_nvfp4 uses) applied to n binary32
 * values: out[i] = E2M1_rne_satfinite(in[i]) in bits 0-3.  Device pointers. */
FP8RL_API fp8rl_status fp8rl_debug_e2m1_encode(const float* in, uint8_t* out, int64_t n,
                                               fp8rl_stream_t stream);

/* Checks the quantizers' division-free encode against IEEE division on the device: for
 * every BF16 group maximum with bits in [amax_lo, amax_hi) (positive finite: below 0x7F80)
 * and every BF16 x with |x| <= amax, both signs, the code of E4M3(fl32(x / s)) with
 * s = fl32(amax / 448) must equal the production encode.  Adds the number of mismatching
 * pairs to *mismatches and stores the first one as (amax_bits << 16) | |x|_bits into
 * *first_bad if that still holds 0xFFFFFFFF.  Device pointers. */
FP8RL_API fp8rl_status fp8rl_debug_encode_check(uint32_t amax_lo, uint32_t amax_hi,
                                                unsigned long long* mismatches,
                                                uint32_t* first_bad, fp8rl_stream_t stream);

/* Launches one CTA that waits, with the GEMM kernels' bounded wait, on an mbarrier that
 * nothing completes; after `timeout_ns` it records FP8RL_ERR_DEVICE_TIMEOUT and returns.
 * Exercises the failure path without faulting or hanging the GPU. */
FP8RL_API fp8rl_status fp8rl_debug_wait_timeout(uint64_t timeout_ns, fp8rl_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8RL_H */
