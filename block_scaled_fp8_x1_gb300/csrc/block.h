// block.h -- launchers of the block operators around the FP8 linears (internal): the fused
// residual + norms and its backward, and SiLU-mul with an 8-bit checkpoint of its input.
#pragma once

#include "gemm.h"

namespace fp8rl {

// residual_norm.cu.  K % 128 == 0, K <= kResNormMaxK.  A saved tensor of the backward is BF16
// (codes null) or E4M3 codes with 1x128 scales s[K/128][M].
constexpr int64_t kResNormMaxK = 8192;

cudaError_t launch_residual_norm(const fp8rl_residual_norm_args& a, int64_t M, int64_t K, int num_sms, cudaStream_t st);
int residual_norm_bwd_blocks(int64_t M, int64_t K, int num_sms);
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

}  // namespace fp8rl
