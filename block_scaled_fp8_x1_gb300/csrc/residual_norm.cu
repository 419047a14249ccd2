// residual_norm.cu -- the norms before and after a block, fused with the block's gate, its
// residual scale, the residual add and the quantizer of the next linear; and the gradients.
//
// Forward, per row (r(v) = 1/sqrt(mean(v^2) + eps), all in FP32):
//     n  = y r(y) g_post                     (n = y without a post norm)
//     h' = bf16(h + alpha gate n)            (gate = 1 without one)
//     z  = bf16((h' r(h')) g_pre)            -> BF16, or E4M3 per 1x128
// and, on request, the 1x128 codes of h' and y for the backward pass.  The statistics of the
// second norm are those of the rounded h', the tensor that the next operator and the backward
// pass see.
//
// Backward.  With x^ = x r and the cotangent t of x^, the gradient of x is
// r (t - x^ mean(t x^)).  So, with dz and dh the gradients of z and h':
//     dH     = dh + r (t - x^ mean(t x^)),  t = dz g_pre,  x^ = h' r        (gradient of h)
//     dn     = alpha gate dH
//     dy     = r_y (u - y^ mean(u y^)),     u = dn g_post, y^ = y r_y       (or dy = dn)
//     dg_pre = sum_m dz x^,  dg_post = sum_m dn y^,  dgate = sum_m alpha dH n
// dH stays in FP32 between the two halves.
#include "block.h"
#include "quant_common.cuh"

namespace fp8rl {

namespace {

__device__ __forceinline__ uint4 ld_v4(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ float elem(const uint4& v, int j) {
    const uint32_t w = (j >> 1) == 0 ? v.x : (j >> 1) == 1 ? v.y : (j >> 1) == 2 ? v.z : v.w;
    return (j & 1) ? bf16_hi(w) : bf16_lo(w);
}

// Sum of one value per thread over the CTA, the same in every thread: a shuffle tree in each
// warp, then one over the warps' sums (buf[w], zero from nwarps up to 32).  Successive calls
// alternate between two buffers: a buffer is written again only after the barrier of the call in
// between, which every reader has reached.
__device__ __forceinline__ float warp_sum(float v) {
    #pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
__device__ __forceinline__ float block_sum(float v, float* buf) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(buf[threadIdx.x & 31]);
}

__device__ __forceinline__ float2 pair(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// Codes of four pairs of a group whose scale is too small for the division-free encode.
__device__ __noinline__ uint2 encode8_slow(uint4 v, float s) {
    uint32_t c[4];
    #pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = e4m3x2(__fdiv_rn(bf16_lo(word(v, j)), s), __fdiv_rn(bf16_hi(word(v, j)), s));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// 1x128 codes of a row: thread t holds 8 columns of BF16 pairs, so a group is 16 lanes.  Every
// lane of the warp takes part.
__device__ __forceinline__ void quant_row(const uint4& v, bool act, uint8_t* q, float* s) {
    uint32_t mx = absmax2(absmax2(absmax2(absmax2(0u, v.x), v.y), v.z), v.w);
    mx = max(mx & 0xFFFFu, mx >> 16);
    #pragma unroll
    for (int off = 8; off >= 1; off >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (!act) return;
    const FastScale f = fast_scale(bf16_bits_amax_to_f32(mx));
    uint2 c = make_uint2(flip_codes(encode_pair_neg(pair(v.x), f.s, f.nr), encode_pair_neg(pair(v.y), f.s, f.nr), f.keep),
                         flip_codes(encode_pair_neg(pair(v.z), f.s, f.nr), encode_pair_neg(pair(v.w), f.s, f.nr), f.keep));
    if (f.slow) c = encode8_slow(v, f.s);
    *reinterpret_cast<uint2*>(q) = c;
    if ((threadIdx.x & 15) == 0) *s = f.s;
}

__device__ __forceinline__ float rstd_of(float sumsq, float k, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sumsq, k), eps)));
}

}  // namespace

// One row per CTA at a time; thread t holds columns 8 (t + NT i), i < NCH.  The next row's words
// are requested before this row is reduced.  The layout depends on K alone, so a token's row has
// the same bits alone and in a batch.
template <bool POST, int NCH>
__global__ void __launch_bounds__(512, 2) k_residual_norm(const fp8rl_residual_norm_args a, int64_t M, int64_t K) {
    extern __shared__ __align__(16) float s_w[];      // alpha * gate * g_post [K]
    __shared__ float s_sum[2][32];
    const int tid = threadIdx.x, nt = blockDim.x;
    const float kf = (float)K;
    int par = 0;
    uint4 pre[NCH];
    #pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = 8 * (tid + nt * i);
        const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        pre[i] = make_uint4(0, 0, 0, 0);
        if (c < K) {
            const uint4 g = a.gate ? ld_v4(a.gate + c) : one;
            const uint4 p = POST ? ld_v4(a.post_gamma + c) : one;
            pre[i] = ld_v4(a.pre_gamma + c);
            #pragma unroll
            for (int j = 0; j < 8; ++j) s_w[c + j] = a.alpha * elem(g, j) * elem(p, j);
        }
    }
    if (tid < 32) s_sum[0][tid] = s_sum[1][tid] = 0.0f;
    __syncthreads();
    uint4 nh[NCH], ny[NCH];
    auto load_row = [&](int64_t m) {
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = 8 * (tid + nt * i);
            nh[i] = ny[i] = make_uint4(0, 0, 0, 0);
            if (c < K && m < M) {
                nh[i] = ld_v4(a.h + m * a.ldh + c);
                ny[i] = ld_v4(a.y + m * a.ldy + c);
            }
        }
    };
    load_row(blockIdx.x);
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        uint4 hv[NCH], yv[NCH];
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            hv[i] = nh[i];
            yv[i] = ny[i];
        }
        load_row(m + gridDim.x);
        float ry = 1.0f;
        if (POST) {
            float2 ss = both(0.0f);
            #pragma unroll
            for (int i = 0; i < NCH; ++i)
                #pragma unroll
                for (int j = 0; j < 4; ++j) ss = __ffma2_rn(pair(word(yv[i], j)), pair(word(yv[i], j)), ss);
            ry = rstd_of(block_sum(ss.x + ss.y, s_sum[par]), kf, a.eps);
            par ^= 1;
        }
        float2 ss = both(0.0f);
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = 8 * (tid + nt * i);
            uint32_t o[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 w = c < K ? *reinterpret_cast<const float2*>(s_w + c + 2 * j) : both(0.0f);
                const float2 x = __ffma2_rn(__fmul2_rn(pair(word(yv[i], j)), both(ry)), w, pair(word(hv[i], j)));
                o[j] = pack_bf16x2(x.x, x.y);
                ss = __ffma2_rn(pair(o[j]), pair(o[j]), ss);
            }
            hv[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        const float r = rstd_of(block_sum(ss.x + ss.y, s_sum[par]), kf, a.eps);
        par ^= 1;
        if (tid == 0) {
            a.r_pre[m] = r;
            if (POST) a.r_post[m] = ry;
        }
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = 8 * (tid + nt * i);
            const bool act = c < K;
            uint32_t o[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = __fmul2_rn(__fmul2_rn(pair(word(hv[i], j)), both(r)), pair(word(pre[i], j)));
                o[j] = pack_bf16x2(x.x, x.y);
            }
            const uint4 z = make_uint4(o[0], o[1], o[2], o[3]);
            if (act) *reinterpret_cast<uint4*>(a.h_out + m * K + c) = hv[i];
            const int64_t sc = (int64_t)(c >> 7) * M + m;
            if (a.z && act) *reinterpret_cast<uint4*>(a.z + m * K + c) = z;
            if (a.q) quant_row(z, act, a.q + m * K + c, a.s + sc);
            if (a.qh) quant_row(hv[i], act, a.qh + m * K + c, a.sh + sc);
            if (a.qy) quant_row(yv[i], act, a.qy + m * K + c, a.sy + sc);
        }
    }
}

static int norm_threads(int64_t K) { return (int)((K / 8 + 31) / 32 * 32); }

template <int NCH>
static cudaError_t launch_fwd_t(const fp8rl_residual_norm_args& a, int64_t M, int64_t K, int num_sms, cudaStream_t st) {
    const int nt = norm_threads((K / 8 + NCH - 1) / NCH * 8);
    auto kern = a.post_gamma ? k_residual_norm<true, NCH> : k_residual_norm<false, NCH>;
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, nt, (size_t)K * 4);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
    kern<<<(unsigned)(M < grid ? M : grid), nt, (size_t)K * 4, st>>>(a, M, K);
    return cudaGetLastError();
}

cudaError_t launch_residual_norm(const fp8rl_residual_norm_args& a, int64_t M, int64_t K, int num_sms, cudaStream_t st) {
    if (K <= 4096) return launch_fwd_t<1>(a, M, K, num_sms, st);
    return launch_fwd_t<2>(a, M, K, num_sms, st);
}

// ------------------------------------------------------------------------------------ backward

namespace {

// Eight saved values: BF16 words, or E4M3 codes times their group's scale.
struct Saved8 {
    uint4 w;      // BF16 pairs, or the eight codes in x, y
    float s;
};
template <bool CK>
__device__ __forceinline__ void saved_values(const Saved8& v, float (&x)[8]) {
    if (!CK) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = elem(v.w, j);
        return;
    }
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint16_t pair = (uint16_t)((j < 2 ? v.w.x : v.w.y) >> (16 * (j & 1)));
        float d0, d1;
        asm("{\n\t.reg .b32 h;\n\t.reg .f16 a, b;\n\t"
            "cvt.rn.f16x2.e4m3x2 h, %2;\n\t"
            "mov.b32 {a, b}, h;\n\t"
            "cvt.f32.f16 %0, a;\n\t"
            "cvt.f32.f16 %1, b;\n\t}"
            : "=f"(d0), "=f"(d1)
            : "h"(pair));
        x[2 * j] = d0 * v.s;
        x[2 * j + 1] = d1 * v.s;
    }
}
template <bool CK>
__device__ __forceinline__ Saved8 load_saved(const uint16_t* x, int64_t ld, const uint8_t* q, const float* s, int64_t m,
                                             int64_t c, int64_t M, int64_t K) {
    Saved8 v;
    v.s = 0.0f;
    if (CK) {
        const uint2 w = *reinterpret_cast<const uint2*>(q + m * K + c);
        v.w = make_uint4(w.x, w.y, 0, 0);
        v.s = s[(c >> 7) * M + m];
    } else {
        v.w = ld_v4(x + m * ld + c);
    }
    return v;
}

}  // namespace

// Row block b of the grid takes rows [b rows, (b+1) rows).  Thread t holds columns 8 (t + NT i),
// i < NCH; its shares of the column sums stay in registers over the rows and go to
// ws[b][0..2][K] (g_pre, g_post, gate), which k_resnorm_colsum adds in block order.
template <bool POST, bool GATE, bool CK, int NCH>
__global__ void __launch_bounds__(NCH == 1 ? 640 : 512, 1)
    k_residual_norm_bwd(const fp8rl_residual_norm_bwd_args a, int64_t M, int64_t K, float* __restrict__ ws) {
    constexpr bool NEED_Y = POST || GATE;
    __shared__ float s_sum[2][32];
    const int tid = threadIdx.x, nt = blockDim.x;
    if (tid < 32) s_sum[0][tid] = s_sum[1][tid] = 0.0f;
    __syncthreads();
    const int64_t rows = (M + gridDim.x - 1) / gridDim.x;
    const int64_t m0 = (int64_t)blockIdx.x * rows;
    const int64_t m1 = m0 + rows < M ? m0 + rows : M;
    const float inv_k = __fdiv_rn(1.0f, (float)K);
    int par = 0;
    uint4 pre[NCH], post[NCH], gate[NCH];
    float a_pre[NCH][8], a_post[NCH][8], a_gate[NCH][8];
    #pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int64_t c = 8 * (int64_t)(tid + nt * i);
        const uint4 zero = make_uint4(0, 0, 0, 0);
        pre[i] = c < K ? ld_v4(a.pre_gamma + c) : zero;
        post[i] = POST && c < K ? ld_v4(a.post_gamma + c) : zero;
        gate[i] = GATE && c < K ? ld_v4(a.gate + c) : zero;
        #pragma unroll
        for (int j = 0; j < 8; ++j) a_pre[i][j] = a_post[i][j] = a_gate[i][j] = 0.0f;
    }
    for (int64_t m = m0; m < m1; ++m) {
        const float r = a.r_pre[m];
        const float ry = POST ? a.r_post[m] : 1.0f;
        uint4 dzv[NCH], dhv[NCH];
        Saved8 hv[NCH], yv[NCH];
        float part = 0.0f;
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int64_t c = 8 * (int64_t)(tid + nt * i);
            dzv[i] = dhv[i] = make_uint4(0, 0, 0, 0);
            hv[i].w = yv[i].w = make_uint4(0, 0, 0, 0);
            hv[i].s = yv[i].s = 0.0f;
            if (c < K) {
                dzv[i] = ld_v4(a.dz + m * a.lddz + c);
                if (a.dh) dhv[i] = ld_v4(a.dh + m * a.lddh + c);
                hv[i] = load_saved<CK>(a.h, a.ldh, a.qh, a.sh, m, c, M, K);
                if (NEED_Y) yv[i] = load_saved<CK>(a.y, a.ldy, a.qy, a.sy, m, c, M, K);
            }
            float x[8];
            saved_values<CK>(hv[i], x);
            #pragma unroll
            for (int j = 0; j < 8; ++j) part = fmaf(elem(dzv[i], j) * elem(pre[i], j), x[j] * r, part);
        }
        const float mean1 = block_sum(part, s_sum[par]) * inv_k;
        par ^= 1;
        float u[NCH][8];
        part = 0.0f;
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int64_t c = 8 * (int64_t)(tid + nt * i);
            float x[8], y[8], dH[8];
            saved_values<CK>(hv[i], x);
            if (NEED_Y) saved_values<CK>(yv[i], y);
            #pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = x[j] * r, dz = elem(dzv[i], j);
                a_pre[i][j] = fmaf(dz, xh, a_pre[i][j]);
                dH[j] = fmaf(r, fmaf(-xh, mean1, dz * elem(pre[i], j)), elem(dhv[i], j));
                float d = a.alpha * dH[j];
                const float yh = NEED_Y ? (POST ? y[j] * ry : y[j]) : 0.0f;
                if (GATE) {
                    a_gate[i][j] = fmaf(d, POST ? yh * elem(post[i], j) : yh, a_gate[i][j]);
                    d *= elem(gate[i], j);
                }
                if (POST) {
                    a_post[i][j] = fmaf(d, yh, a_post[i][j]);
                    d *= elem(post[i], j);
                    part = fmaf(d, yh, part);
                }
                u[i][j] = d;
            }
            if (c < K)
                *reinterpret_cast<uint4*>(a.dh_out + m * K + c) =
                    make_uint4(pack_bf16x2(dH[0], dH[1]), pack_bf16x2(dH[2], dH[3]), pack_bf16x2(dH[4], dH[5]),
                               pack_bf16x2(dH[6], dH[7]));
        }
        float mean2 = 0.0f;
        if (POST) {
            mean2 = block_sum(part, s_sum[par]) * inv_k;
            par ^= 1;
        }
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int64_t c = 8 * (int64_t)(tid + nt * i);
            if (POST) {
                float y[8];
                saved_values<CK>(yv[i], y);
                #pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] = ry * fmaf(-(y[j] * ry), mean2, u[i][j]);
            }
            if (c < K)
                *reinterpret_cast<uint4*>(a.dy + m * K + c) =
                    make_uint4(pack_bf16x2(u[i][0], u[i][1]), pack_bf16x2(u[i][2], u[i][3]),
                               pack_bf16x2(u[i][4], u[i][5]), pack_bf16x2(u[i][6], u[i][7]));
        }
    }
    #pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int64_t c = 8 * (int64_t)(tid + nt * i);
        if (c >= K) continue;
        float* dst = ws + (int64_t)blockIdx.x * 3 * K + c;
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            dst[j] = a_pre[i][j];
            if (POST) dst[K + j] = a_post[i][j];
            if (GATE) dst[2 * K + j] = a_gate[i][j];
        }
    }
}

// Column sums over the row blocks: 32 columns by 8 slices of the blocks per CTA, each slice in
// block order, then the slices in order.
__global__ void __launch_bounds__(256) k_resnorm_colsum(const float* __restrict__ ws, int nblocks, int64_t K,
                                                        float* dpre, float* dpost, float* dgate) {
    __shared__ float part[8][33];
    const int x = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t k = (int64_t)blockIdx.x * 32 + x;
    float* out = blockIdx.y == 0 ? dpre : blockIdx.y == 1 ? dpost : dgate;
    if (!out) return;
    float s = 0.0f;
    for (int b = sl; b < nblocks; b += 8) s += ws[((int64_t)b * 3 + blockIdx.y) * K + k];
    part[sl][x] = s;
    __syncthreads();
    if (sl == 0) {
        for (int i = 1; i < 8; ++i) s += part[i][x];
        out[k] = s;
    }
}

static int bwd_nch(int64_t K) { return K <= 8 * 640 ? 1 : 2; }

int residual_norm_bwd_blocks(int64_t M, int64_t K, int num_sms) {
    const int nch = bwd_nch(K);
    const int nt = norm_threads((K / nch + 127) / 128 * 128);
    int per = (nch == 1 ? 640 : 512) / nt;
    if (per > 8) per = 8;
    if (per < 1) per = 1;
    const int64_t b = (int64_t)num_sms * per;
    return (int)(M < b ? M : b);
}

template <bool POST, bool GATE, bool CK>
static cudaError_t launch_bwd_t(const fp8rl_residual_norm_bwd_args& a, int64_t M, int64_t K, float* ws, int nb,
                                cudaStream_t st) {
    const int nch = bwd_nch(K);
    const int nt = norm_threads((K / nch + 127) / 128 * 128);
    if (nch == 1) k_residual_norm_bwd<POST, GATE, CK, 1><<<nb, nt, 0, st>>>(a, M, K, ws);
    else k_residual_norm_bwd<POST, GATE, CK, 2><<<nb, nt, 0, st>>>(a, M, K, ws);
    return cudaGetLastError();
}

cudaError_t launch_residual_norm_bwd(const fp8rl_residual_norm_bwd_args& a, int64_t M, int64_t K, float* ws,
                                     int nblocks, cudaStream_t st) {
    const bool ck = a.qh != nullptr;
    cudaError_t e;
    if (a.post_gamma) {
        if (a.gate) e = ck ? launch_bwd_t<true, true, true>(a, M, K, ws, nblocks, st) : launch_bwd_t<true, true, false>(a, M, K, ws, nblocks, st);
        else e = ck ? launch_bwd_t<true, false, true>(a, M, K, ws, nblocks, st) : launch_bwd_t<true, false, false>(a, M, K, ws, nblocks, st);
    } else {
        if (a.gate) e = ck ? launch_bwd_t<false, true, true>(a, M, K, ws, nblocks, st) : launch_bwd_t<false, true, false>(a, M, K, ws, nblocks, st);
        else e = ck ? launch_bwd_t<false, false, true>(a, M, K, ws, nblocks, st) : launch_bwd_t<false, false, false>(a, M, K, ws, nblocks, st);
    }
    if (e != cudaSuccess) return e;
    k_resnorm_colsum<<<dim3((unsigned)(K / 32), 3, 1), 256, 0, st>>>(ws, nblocks, K, a.dpre,
                                                                    a.post_gamma ? a.dpost : nullptr,
                                                                    a.gate ? a.dgate : nullptr);
    return cudaGetLastError();
}

}  // namespace fp8rl
