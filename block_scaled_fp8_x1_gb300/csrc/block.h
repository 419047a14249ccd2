// block.h -- launchers of the block operators around the FP8 linears (internal): the fused
// residual + norms and its backward, SiLU-mul with an 8-bit checkpoint of its input, and the
// product of a few tokens with NVFP4 weights.
#pragma once

#include "gemm.h"

namespace fp8rl {

// residual_norm.cu.  K % 128 == 0, K <= kResNormMaxK.  A saved tensor of the backward is BF16
// (codes null) or E4M3 codes with 1x128 scales s[K/128][M].
constexpr int64_t kResNormMaxK = 8192;

cudaError_t launch_residual_norm(const fp8rl_residual_norm_args& a, int64_t M, int64_t K, int num_sms, cudaStream_t st);
// Row blocks of the backward; a row of checkpoints takes less shared memory, so no form has more
// blocks than that one.
int residual_norm_bwd_blocks(int64_t M, int64_t K, bool ckpt, int num_sms);
cudaError_t launch_residual_norm_bwd(const fp8rl_residual_norm_bwd_args& a, int64_t M, int64_t K, float* ws,
                                     int nblocks, cudaStream_t st);

// quantize.cu: the 128x1 codes of z = bf16((x * rstd) * gamma) from a given rstd.
cudaError_t launch_rmsnorm_cols(const uint16_t* x, const uint16_t* gamma, const float* rstd, int64_t M, int64_t K,
                                uint8_t* qT, float* sT, uint64_t timeout_ns, cudaStream_t st);

// quantize.cu: SiLU-mul -> quantize that also writes the 1x128 codes of gu (the checkpoint),
// and its backward from them.
cudaError_t launch_silu_mul_quant_ckpt(const uint16_t* gu, int64_t M, int64_t I, uint8_t* q, float* s, uint8_t* qT,
                                       float* sT, uint8_t* qgu, float* sgu, uint64_t timeout_ns, cudaStream_t st);
cudaError_t launch_silu_mul_bwd_quant_ckpt(const uint8_t* qgu, const float* sgu, const uint16_t* dh, int64_t M, int64_t I,
                                           uint8_t* q, float* s, uint8_t* qT, float* sT, uint64_t timeout_ns,
                                           cudaStream_t st);

// matvec.cu: y = x W^T for M <= 16 BF16 tokens, W in NVFP4 (codes, scale atoms, row scales).
struct MatvecParams {
    int M;                   // tokens, 1..16
    bool one;                // the one-token form (M == 1)
    int nkb;                 // K / 128 (even)
    int tiles;               // N / 32 (a multiple of 4)
    int splits;              // CTAs of a cluster that share K, 1..8
    int wk;                  // warps of a CTA that share K: 1, 2, 4, 8 or 16
    const uint16_t* x;
    int64_t ldx;
    const uint8_t* qw;
    const uint8_t* sfw;
    const float* gw;
    uint16_t* y;
    int64_t ldy;
};
constexpr int kMatvecMaxTokens = 16;
constexpr int kMatvecWarps = 16;
constexpr size_t kMatvecMaxSmem = 224 * 1024;
size_t matvec_smem(int M, int nkb, int splits, bool one);   // dynamic shared memory of a CTA
// `clusters` of p.splits CTAs, each taking every clusters-th group of kMatvecWarps / wk tiles of
// 32 rows.
cudaError_t launch_matvec_nvfp4(const MatvecParams& p, int clusters, cudaStream_t st);

}  // namespace fp8rl
