// experts.h -- launchers of the expert-layer operators (internal): the router, the sort of
// (token, expert) pairs, the gather / combine between token and expert order, and the products of
// every expert's rows with its own weight matrix.
#pragma once

#include "gemm.h"

namespace fp8rl {

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxTopK = 32;
constexpr int64_t kMaxGroups = 32;
constexpr int64_t kMaxPairs = int64_t(1) << 30;
constexpr int64_t kMaxCombineColumns = int64_t(1) << 24;
constexpr int64_t kExpertAlign = 128;   // the row alignment that the training forms need

// route.cu
cudaError_t launch_route_topk(const fp8rl_route_args& a, int64_t T, int64_t E, cudaStream_t st);
cudaError_t launch_route_topk_bwd(const fp8rl_route_bwd_args& a, int64_t T, int64_t E, cudaStream_t st);

// expert_rows.cu.  Blocks of the sort: the workspace holds a histogram of E counts for each when
// there are several.
int expert_rows_blocks(int64_t P);
cudaError_t launch_expert_rows(const int32_t* index, int64_t P, int E, int align, int64_t R, int32_t* pos, int32_t* src,
                               int32_t* start, int32_t* count, int32_t* hist, cudaStream_t st);
cudaError_t launch_expert_combine(const uint16_t* y, int64_t ldy, int64_t N, const float* weight, const uint16_t* residual,
                                  int64_t ldr, const fp8rl_expert_layout& l, uint16_t* out, int64_t ldo, cudaStream_t st);
cudaError_t launch_expert_dweight(const uint16_t* dout, int64_t ldd, const uint16_t* y, int64_t ldy, int64_t N,
                                  const fp8rl_expert_layout& l, float* dweight, cudaStream_t st);

// quantize.cu: the gathered rows quantized 1x128 and, with qT, 128x1 (l.R % 128 == 0 then).
cudaError_t launch_expert_gather(const uint16_t* x, int64_t ldx, int64_t K, const float* weight, const fp8rl_expert_layout& l,
                                 uint8_t* q, float* s, uint8_t* qT, float* sT, int num_sms, cudaStream_t st);

// gemm_experts.cu: the paired-SM GEMM over the experts' row segments (aligned to 128).
enum ExpertOp : int { EXPERT_FWD = 0, EXPERT_DGRAD = 1, EXPERT_WGRAD = 2 };
struct ExpertGemmParams {
    const int32_t* start;    // [E + 1]
    int E;
    int R;                   // rows of the layout
    int rows;                // WGRAD: rows of one expert's result (N); else unused
    int cols;                // columns of the result
    int nkb;                 // FWD, DGRAD: K-blocks of the reduction (WGRAD: each expert's own rows)
    int b_x, b_y;            // FWD, DGRAD: expert e's B starts at coordinates (e * b_x, e * b_y)
    const float* sb;         // FWD, DGRAD: block scales sb[e * sb_e + column block * sb_c + kb * sb_kb]
    int64_t sb_e, sb_c, sb_kb;
    uint64_t timeout_ns;
};
cudaError_t launch_gemm_experts(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tsa, const CUtensorMap& tsb,
                                const CUtensorMap& tc, const ExpertGemmParams& p, bool wgrad, int clusters, cudaStream_t st);
fp8rl_status read_and_clear_experts_status();

// decode_experts.cu: a few tokens an expert, weights on the MMA's M side.
struct ExpertDecodeParams {
    const int32_t* start;    // [E + 1]
    const int32_t* count;    // [E]
    int E;
    int nkb;                 // K / 128
    int tiles;               // N / 128
    int max_items;           // (unit, tile) items of any counts that fit the rows
    const float* sx;         // sx[kb * R + r]
    int64_t R;
    const float* sw;         // sw[(e * tiles + tile) * nkb + kb]
    uint16_t* y;             // y[r * ldy + n]
    int64_t ldy;
    uint64_t timeout_ns;
};
int expert_decode_tokens(int64_t P, int64_t E);                    // token rows of a tile
int expert_decode_splits(int64_t items, int64_t nkb, int num_sms);  // CTAs of a cluster
// `clusters` of `splits` CTAs: one for every item there can be when splits > 1, else any number.
cudaError_t launch_decode_experts(const CUtensorMap& tw, const CUtensorMap& tx, const ExpertDecodeParams& p, int tokens,
                                  int clusters, int splits, cudaStream_t st);
fp8rl_status read_and_clear_decode_experts_status();

}  // namespace fp8rl
