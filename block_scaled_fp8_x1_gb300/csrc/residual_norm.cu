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
//
// What bounds them.  The forward moves 6 bytes an element in and out for h, y, h' and 1 to 2 more
// for each form of z and each checkpoint: 16384 x 5120 to BF16 takes 102 us, 0.97 of the measured
// copy rate; with z's codes and both checkpoints 153 us (0.74), with 63% of the issue slots used: the
// three encodes are dependent chains and 20 warps an SM do not fill their gaps; and the 128x1 codes, a second kernel that reads h' again, 58 us more.  The
// backward of the same size takes 158 us from BF16 (0.94) and 151 us from checkpoints (0.83).
#include "block.h"
#include "quant_common.cuh"

namespace fp8rl {

namespace {

__device__ __forceinline__ uint4 ld_v4(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

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

// Largest |BF16| of eight values, per half of the word.
__device__ __forceinline__ uint32_t max8(const uint4& v) { return absmax2(absmax2(absmax2(absmax2(0u, v.x), v.y), v.z), v.w); }

// 1x128 codes of G groups of 128 that a half-warp holds, 8 values a lane and group.  The maxima
// are reduced two to a word; lane g of the half-warp forms the scale of group g, once, stores it
// at sp (null: a group that is not written), and hands it to the others.  Every lane of the warp
// takes part; `codes` gets the eight codes of each group.
template <int G>
__device__ __forceinline__ void quant_groups(const uint4 (&v)[G], float* sp, uint2 (&codes)[G]) {
    const int lane = threadIdx.x & 31, me = lane & 15;
    uint32_t mx[(G + 1) / 2];
    #pragma unroll
    for (int g = 0; g < G; g += 2) {
        const uint32_t w0 = max8(v[g]), w1 = g + 1 < G ? max8(v[g + 1 < G ? g + 1 : g]) : 0u;
        uint32_t m = __vmaxu2(__byte_perm(w0, w1, 0x5410), __byte_perm(w0, w1, 0x7632));
        #pragma unroll
        for (int off = 8; off >= 1; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
        mx[g / 2] = m;
    }
    uint32_t mine = mx[0];
    #pragma unroll
    for (int i = 1; i < (G + 1) / 2; ++i) mine = (me >> 1) == i ? mx[i] : mine;
    const FastScale f = fast_scale(bf16_bits_amax_to_f32((me & 1) ? mine >> 16 : mine & 0xFFFFu));
    if (sp) *sp = f.s;
    const bool slow = __any_sync(0xffffffffu, me < G && f.slow);
    #pragma unroll
    for (int g = 0; g < G; ++g) {
        const float sg = __shfl_sync(0xffffffffu, f.s, (lane & 16) | g), nr = __shfl_sync(0xffffffffu, f.nr, (lane & 16) | g);
        const uint32_t keep = sg == 0.0f ? 0u : 0xFFFFFFFFu;
        codes[g] = make_uint2(flip_codes(encode_pair_neg(pair(v[g].x), sg, nr), encode_pair_neg(pair(v[g].y), sg, nr), keep),
                              flip_codes(encode_pair_neg(pair(v[g].z), sg, nr), encode_pair_neg(pair(v[g].w), sg, nr), keep));
        if (slow && sg > 0.0f && scale_is_slow(sg)) codes[g] = encode8_slow(v[g], sg);
    }
}

// 1/sqrt(mean + eps): the hardware's reciprocal square root r (2 ulp) and one step of Newton's method,
// r + r (1 - v r^2) / 2, with the rounding error of v r in the residual, so that the result is v's
// root rounded once (without it, off by up to one unit in the last place).  Infinite or zero v keeps the
// first value.
__device__ __forceinline__ float rstd_of(float sumsq, float inv_k, float eps) {
    const float v = fmaf(sumsq, inv_k, eps), r = rsqrtf(v), p = __fmul_rn(v, r);
    const float e = fmaf(-fmaf(v, r, -p), r, fmaf(-p, r, 1.0f));
    return fabsf(e) < 1.0f ? fmaf(0.5f * r, e, r) : r;
}

}  // namespace

// One row per CTA at a time; thread t holds columns 8 (t + NT i), i < NCH.  The next row's words
// are requested before this row is reduced.  The layout depends on K alone, so a token's row has
// the same bits alone and in a batch.  Q: z is quantized; CK: h' or y or both are.
template <bool POST, bool Q, bool CK, int NCH, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k_residual_norm(const fp8rl_residual_norm_args a, int64_t M, int64_t K) {
    grid_dependency_begin();
    // gate * g_post (exact: two BF16 factors), [NCH][4 pairs][threads]; alpha is multiplied in last, so
    // that without a post norm the branch takes the one rounding of alpha (gate y)
    extern __shared__ __align__(16) float2 s_w[];
    __shared__ float s_sum[2][32];
    const int tid = threadIdx.x, nt = blockDim.x, me = tid & 15;
    const float inv_k = __fdiv_rn(1.0f, (float)K);
    int par = 0;
    uint4 pre[NCH];
    #pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = 8 * (tid + nt * i);
        const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), zero = make_uint4(0, 0, 0, 0);
        const uint4 g = c < K ? (a.gate ? ld_v4(a.gate + c) : one) : zero;
        const uint4 p = c < K && POST ? ld_v4(a.post_gamma + c) : one;
        pre[i] = c < K ? ld_v4(a.pre_gamma + c) : zero;
        #pragma unroll
        for (int j = 0; j < 4; ++j)
            s_w[(i * 4 + j) * nt + tid] = __fmul2_rn(pair(word(g, j)), pair(word(p, j)));
    }
    if (tid < 32) s_sum[0][tid] = s_sum[1][tid] = 0.0f;
    // groups of a half-warp: z's chunks, then h's, then y's; lane `me` stores the scale of group me
    constexpr int G = NCH * ((Q ? 1 : 0) + (CK ? 2 : 0));
    float* sp = nullptr;
    if (me < G) {
        const int which = me / NCH + (Q ? 0 : 1);
        const int64_t c = 8 * (int64_t)((tid & ~15) + nt * (me % NCH));
        float* s = which == 0 ? a.s : which == 1 ? a.sh : a.sy;
        if (s && c < K) sp = s + (c >> 7) * M;
    }
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
            ry = rstd_of(block_sum(ss.x + ss.y, s_sum[par]), inv_k, a.eps);
            par ^= 1;
        }
        float2 ss = both(0.0f);
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            uint32_t o[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 y = POST ? __fmul2_rn(pair(word(yv[i], j)), both(ry)) : pair(word(yv[i], j));
                const float2 x = __fadd2_rn(__fmul2_rn(__fmul2_rn(y, s_w[(i * 4 + j) * nt + tid]), both(a.alpha)), pair(word(hv[i], j)));
                o[j] = pack_bf16x2(x.x, x.y);
                ss = __ffma2_rn(pair(o[j]), pair(o[j]), ss);
            }
            hv[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        const float r = rstd_of(block_sum(ss.x + ss.y, s_sum[par]), inv_k, a.eps);
        par ^= 1;
        if (tid == 0) {
            a.r_pre[m] = r;
            if (POST) a.r_post[m] = ry;
        }
        uint4 z[NCH];
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = 8 * (tid + nt * i);
            uint32_t o[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = __fmul2_rn(__fmul2_rn(pair(word(hv[i], j)), both(r)), pair(word(pre[i], j)));
                o[j] = pack_bf16x2(x.x, x.y);
            }
            z[i] = make_uint4(o[0], o[1], o[2], o[3]);
            if (c < K) {
                *reinterpret_cast<uint4*>(a.h_out + m * K + c) = hv[i];
                if (a.z) *reinterpret_cast<uint4*>(a.z + m * K + c) = z[i];
            }
        }
        if constexpr (G > 0) {
            uint4 v[G];
            uint2 codes[G];
            #pragma unroll
            for (int g = 0; g < G; ++g) {
                const int which = g / NCH + (Q ? 0 : 1), i = g % NCH;
                v[g] = which == 0 ? z[i] : which == 1 ? hv[i] : yv[i];
            }
            quant_groups<G>(v, sp ? sp + m : nullptr, codes);
            #pragma unroll
            for (int g = 0; g < G; ++g) {
                const int which = g / NCH + (Q ? 0 : 1), c = 8 * (tid + nt * (g % NCH));
                uint8_t* q = which == 0 ? a.q : which == 1 ? a.qh : a.qy;
                if (c < K && (which == 0 || q)) *reinterpret_cast<uint2*>(q + m * K + c) = codes[g];
            }
        }
    }
}

static int norm_threads(int64_t K) { return (int)((K / 8 + 31) / 32 * 32); }

template <bool POST, int NCH, int MAXT, int MINB>
static cudaError_t launch_fwd_t(const fp8rl_residual_norm_args& a, int64_t M, int64_t K, int num_sms, cudaStream_t st) {
    const int nt = norm_threads((K / 8 + NCH - 1) / NCH * 8);
    const bool ck = a.qh || a.qy;
    auto kern = a.q ? (ck ? k_residual_norm<POST, true, true, NCH, MAXT, MINB> : k_residual_norm<POST, true, false, NCH, MAXT, MINB>)
                    : (ck ? k_residual_norm<POST, false, true, NCH, MAXT, MINB> : k_residual_norm<POST, false, false, NCH, MAXT, MINB>);
    const size_t smem = (size_t)nt * NCH * 32;
    int per_sm = 0;
    cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, nt, smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
    return launch_dependent(kern, dim3((unsigned)(M < grid ? M : grid)), dim3(nt), smem, st, a, M, K);
}

template <int NCH, int MAXT, int MINB>
static cudaError_t launch_fwd(const fp8rl_residual_norm_args& a, int64_t M, int64_t K, int num_sms, cudaStream_t st) {
    return a.post_gamma ? launch_fwd_t<true, NCH, MAXT, MINB>(a, M, K, num_sms, st)
                        : launch_fwd_t<false, NCH, MAXT, MINB>(a, M, K, num_sms, st);
}

cudaError_t launch_residual_norm(const fp8rl_residual_norm_args& a, int64_t M, int64_t K, int num_sms, cudaStream_t st) {
    // Two chunks of 8 columns a thread, as many CTAs on an SM as registers allow without spills
    // (the compiler's bound is for the widest row of each range).  16384 x 5120, BF16 out /
    // quantized with both checkpoints, in us: 103 / 153 so, 117 / 166 with three CTAs at 64
    // registers, 102 / 202 with one chunk and 640 threads, 114 / 172 with four chunks.
    if (K <= 2560) return launch_fwd<2, 160, 4>(a, M, K, num_sms, st);
    if (K <= 4096) return launch_fwd<2, 256, 3>(a, M, K, num_sms, st);
    if (K <= 5120) return launch_fwd<2, 320, 2>(a, M, K, num_sms, st);
    return launch_fwd<2, 512, 1>(a, M, K, num_sms, st);
}

// ------------------------------------------------------------------------------------ backward

namespace {

// One row's words of a thread's chunk of 8 columns, as they lie in its slot of shared memory:
// dz and dh (BF16), then h' and y (BF16, or E4M3 codes).  A thread copies
// and reads only its own chunks, so the copies need no barrier, only its own wait.
template <bool CK>
struct Slot {
    static constexpr int SAVED = CK ? 8 : 16;
    static constexpr int BYTES = 32 + 2 * SAVED;   // a chunk of one thread
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Two E4M3 codes to FP32, exactly: through FP16, which holds every finite E4M3.
__device__ __forceinline__ float2 e4m3_pair(uint32_t codes) {
    float2 d;
    asm("{\n\t.reg .b32 h;\n\t.reg .f16 a, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 h, %2;\n\t"
        "mov.b32 {a, b}, h;\n\t"
        "cvt.f32.f16 %0, a;\n\t"
        "cvt.f32.f16 %1, b;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "h"((uint16_t)codes));
    return d;
}

// Eight saved values times f (a checkpoint's scale is in f).
template <bool CK>
__device__ __forceinline__ void saved_times(uint32_t words, float f, float2 (&x)[4]) {
    if (CK) {
        const uint2 c = lds_v2(words);
        const float2 k = both(f);
        #pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(e4m3_pair((j < 2 ? c.x : c.y) >> (16 * (j & 1))), k);
    } else {
        const uint4 w = lds_v4(words);
        #pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(pair(word(w, j)), both(f));
    }
}

}  // namespace

// Row block b of the grid takes rows [b rows, (b+1) rows); thread t holds columns 8 (t + NT i),
// i < NCH.  The rows ahead (SLOTS - 1 of them) are copied to shared memory meanwhile.
//
// With w = alpha gate g_post, u = w dH and v = dH y^: mean(u y^) = mean(w v), and the two column
// sums over the branch are multiples of one, V = sum_m v: dgate = alpha g_post V and
// dg_post = alpha gate V.  So a thread keeps two sums for a column, dg_pre and V, in registers over
// its rows; ws[b][0..1][K] takes them, and k_resnorm_colsum adds the blocks in order.  The sums are
// plain FP32 (error terms would be 16 registers more a thread, past what 640 threads have): a block
// has M / 152 rows or fewer, so a chain grows with M, by 2^-24 of its terms' magnitudes a row at most.
template <bool POST, bool GATE, bool CK, int NCH>
__global__ void __launch_bounds__(NCH == 1 ? 640 : 512, 1)
    k_residual_norm_bwd(const fp8rl_residual_norm_bwd_args a, int64_t M, int64_t K, int slots, float* __restrict__ ws) {
    grid_dependency_begin();
    constexpr bool NEED_Y = POST || GATE;
    using SL = Slot<CK>;
    extern __shared__ __align__(16) uint8_t rn_smem[];
    __shared__ float s_sum[2][32];
    const int tid = threadIdx.x, nt = blockDim.x;
    if (tid < 32) s_sum[0][tid] = s_sum[1][tid] = 0.0f;
    const int64_t rows = (M + gridDim.x - 1) / gridDim.x;
    const int64_t m0 = (int64_t)blockIdx.x * rows;
    const int64_t m1 = m0 + rows < M ? m0 + rows : M;
    const float inv_k = __fdiv_rn(1.0f, (float)K);
    int par = 0;
    // slot layout: for each chunk index i, arrays over the threads of dz, dh, h', y
    const uint32_t base = smem_u32(rn_smem);
    const uint32_t chunk = (uint32_t)nt * SL::BYTES, slot_bytes = chunk * NCH;
    auto at = [&](int slot, int i, int what) -> uint32_t {   // 0 dz, 1 dh, 2 h', 3 y
        const uint32_t b = base + (uint32_t)slot * slot_bytes + (uint32_t)i * chunk;
        if (what < 2) return b + (uint32_t)(what * nt + tid) * 16u;
        return b + (uint32_t)nt * 32u + (uint32_t)((what - 2) * nt + tid) * SL::SAVED;
    };
    auto copy_row = [&](int64_t m, int slot) {
        if (m < m1) {
            #pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int64_t c = 8 * (int64_t)(tid + nt * i);
                if (c >= K) continue;
                cp_async_16(at(slot, i, 0), a.dz + m * a.lddz + c);
                if (a.dh) cp_async_16(at(slot, i, 1), a.dh + m * a.lddh + c);
                if (CK) {
                    cp_async_8(at(slot, i, 2), a.qh + m * K + c);
                    if (NEED_Y) cp_async_8(at(slot, i, 3), a.qy + m * K + c);
                } else {
                    cp_async_16(at(slot, i, 2), a.h + m * a.ldh + c);
                    if (NEED_Y) cp_async_16(at(slot, i, 3), a.y + m * a.ldy + c);
                }
            }
        }
        cp_async_commit();
    };
    // a thread's chunks past K, and dh where there is none, stay zero
    for (int sl = 0; sl < slots; ++sl)
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const bool in = 8 * (int64_t)(tid + nt * i) < K;
            if (!in || !a.dh) st_shared_v4(at(sl, i, 1), make_uint4(0, 0, 0, 0));
            if (!in) {
                st_shared_v4(at(sl, i, 0), make_uint4(0, 0, 0, 0));
                #pragma unroll
                for (int w = 2; w < 4; ++w)
                    #pragma unroll
                    for (int o = 0; o < SL::SAVED; o += 4) st_shared_b32(at(sl, i, w) + o, 0);
            }
        }
    for (int sl = 0; sl < slots - 1; ++sl) copy_row(m0 + sl, sl);

    uint4 pre[NCH];
    float2 w[NCH][4], a_pre[NCH][4], a_v[NCH][4];
    #pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int64_t c = 8 * (int64_t)(tid + nt * i);
        const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        pre[i] = c < K ? ld_v4(a.pre_gamma + c) : make_uint4(0, 0, 0, 0);
        const uint4 p = POST && c < K ? ld_v4(a.post_gamma + c) : one;
        const uint4 g = GATE && c < K ? ld_v4(a.gate + c) : one;
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[i][j] = __fmul2_rn(both(a.alpha), __fmul2_rn(pair(word(g, j)), pair(word(p, j))));   // the inner product is exact
            a_pre[i][j] = a_v[i][j] = both(0.0f);
        }
    }
    // the next row's statistics and the checkpoints' scales, one row ahead in registers
    float r_next = 0.0f, ry_next = 1.0f, sh_next[NCH], sy_next[NCH];
    auto load_scales = [&](int64_t m) {
        if (m >= m1) return;
        r_next = a.r_pre[m];
        if (POST) ry_next = a.r_post[m];
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int64_t c = 8 * (int64_t)(tid + nt * i);
            if (CK && c < K) {
                sh_next[i] = a.sh[(c >> 7) * M + m];
                if (NEED_Y) sy_next[i] = a.sy[(c >> 7) * M + m];
            }
        }
    };
    #pragma unroll
    for (int i = 0; i < NCH; ++i) sh_next[i] = sy_next[i] = CK ? 0.0f : 1.0f;
    load_scales(m0);
    __syncthreads();   // s_sum is zero
    int slot = 0;
    for (int64_t m = m0; m < m1; ++m) {
        const float r = r_next, ry = ry_next;
        float sh[NCH], sy[NCH];
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            sh[i] = sh_next[i] * r;
            sy[i] = POST ? sy_next[i] * ry : sy_next[i];
        }
        load_scales(m + 1);
        // this row's copies have landed when at most the slots - 2 later ones are in flight
        if (slots == 4) cp_async_wait_group<2>();
        else cp_async_wait_group<1>();
        float2 x[NCH][4], t[NCH][4], part = both(0.0f);
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            saved_times<CK>(at(slot, i, 2), sh[i], x[i]);
            const uint4 dz = lds_v4(at(slot, i, 0));
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = pair(word(dz, j));
                t[i][j] = __fmul2_rn(d, pair(word(pre[i], j)));
                part = __ffma2_rn(t[i][j], x[i][j], part);
                a_pre[i][j] = __ffma2_rn(d, x[i][j], a_pre[i][j]);
            }
        }
        const float mean1 = block_sum(part.x + part.y, s_sum[par]) * inv_k;
        par ^= 1;
        // every thread is past the row before: its slot takes the row slots - 1 ahead
        copy_row(m + slots - 1, slot == 0 ? slots - 1 : slot - 1);
        float2 y[NCH][4];
        part = both(0.0f);
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int64_t c = 8 * (int64_t)(tid + nt * i);
            const uint4 dh = lds_v4(at(slot, i, 1));
            if (NEED_Y) saved_times<CK>(at(slot, i, 3), sy[i], y[i]);
            uint32_t o[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 dH = __ffma2_rn(both(r), __ffma2_rn(x[i][j], both(-mean1), t[i][j]), pair(word(dh, j)));
                o[j] = pack_bf16x2(dH.x, dH.y);
                t[i][j] = __fmul2_rn(dH, w[i][j]);
                if (NEED_Y) {
                    const float2 v = __fmul2_rn(dH, y[i][j]);
                    a_v[i][j] = __fadd2_rn(a_v[i][j], v);
                    if (POST) part = __ffma2_rn(v, w[i][j], part);
                }
            }
            if (c < K) *reinterpret_cast<uint4*>(a.dh_out + m * K + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        float mean2 = 0.0f;
        if (POST) {
            mean2 = block_sum(part.x + part.y, s_sum[par]) * inv_k;
            par ^= 1;
        }
        #pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int64_t c = 8 * (int64_t)(tid + nt * i);
            uint32_t o[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 d = t[i][j];
                if (POST) d = __fmul2_rn(both(ry), __ffma2_rn(y[i][j], both(-mean2), d));
                o[j] = pack_bf16x2(d.x, d.y);
            }
            if (c < K) *reinterpret_cast<uint4*>(a.dy + m * K + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        slot = slot + 1 == slots ? 0 : slot + 1;
    }
    cp_async_wait_all();
    #pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int64_t c = 8 * (int64_t)(tid + nt * i);
        if (c >= K) continue;
        float* dst = ws + (int64_t)blockIdx.x * 2 * K + c;
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<float2*>(dst + 2 * j) = a_pre[i][j];
            if (NEED_Y) *reinterpret_cast<float2*>(dst + K + 2 * j) = a_v[i][j];
        }
    }
}

// Column sums over the row blocks: 32 columns by 8 slices of the blocks per CTA, each slice in
// block order, then the slices in order.
__global__ void __launch_bounds__(256) k_resnorm_colsum(const fp8rl_residual_norm_bwd_args a, const float* __restrict__ ws,
                                                        int nblocks, int64_t K) {
    grid_dependency_begin();   // set up as the row kernel ends; its sums are visible from here on
    __shared__ float part[8][33];
    const int x = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t k = (int64_t)blockIdx.x * 32 + x;
    float s = 0.0f;
    #pragma unroll 8
    for (int b = sl; b < nblocks; b += 8) s += ws[((int64_t)b * 2 + blockIdx.y) * K + k];
    part[sl][x] = s;
    __syncthreads();
    if (sl != 0) return;
    for (int i = 1; i < 8; ++i) s += part[i][x];
    if (blockIdx.y == 0) {
        a.dpre[k] = s;
        return;
    }
    const float p = a.post_gamma ? bf16_bits_to_f32(a.post_gamma[k]) : 1.0f;
    const float g = a.gate ? bf16_bits_to_f32(a.gate[k]) : 1.0f;
    if (a.post_gamma) a.dpost[k] = a.alpha * g * s;
    if (a.gate) a.dgate[k] = a.alpha * p * s;
}

// Launch shape: one chunk of 8 columns a thread up to 640 threads (two above, whose sums and
// constants would not fit the registers of 1024 threads), the ring's slots, CTAs per SM.
struct BwdShape {
    int nch, nt, slots, per_sm;
    size_t smem;
};
constexpr int kBwdMaxSmem = 200 * 1024;
static BwdShape bwd_shape(int64_t K, bool ck) {
    BwdShape s;
    s.nch = K <= 8 * 640 ? 1 : 2;
    s.nt = norm_threads((K / 8 + s.nch - 1) / s.nch * 8);
    const size_t row = (size_t)s.nt * s.nch * (ck ? Slot<true>::BYTES : Slot<false>::BYTES);
    s.slots = 4 * row <= kBwdMaxSmem ? 4 : 3;   // 8192 columns of BF16: 3 x 64 KB
    s.smem = (size_t)s.slots * row;
    s.per_sm = (s.nch == 1 ? 640 : 512) / s.nt;
    const int by_smem = (int)(216 * 1024 / (s.smem + 1536));
    if (s.per_sm > by_smem) s.per_sm = by_smem;
    if (s.per_sm > 8) s.per_sm = 8;
    if (s.per_sm < 1) s.per_sm = 1;
    return s;
}

int residual_norm_bwd_blocks(int64_t M, int64_t K, bool ckpt, int num_sms) {
    const int64_t b = (int64_t)num_sms * bwd_shape(K, ckpt).per_sm;
    return (int)(M < b ? M : b);
}

template <bool POST, bool GATE, bool CK>
static cudaError_t launch_bwd_t(const fp8rl_residual_norm_bwd_args& a, int64_t M, int64_t K, float* ws, int nb,
                                cudaStream_t st) {
    const BwdShape s = bwd_shape(K, CK);
    auto kern = s.nch == 1 ? k_residual_norm_bwd<POST, GATE, CK, 1> : k_residual_norm_bwd<POST, GATE, CK, 2>;
    // one limit for every call: host threads may launch different sizes at once
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(nb), dim3(s.nt), s.smem, st, a, M, K, s.slots, ws);
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
    return launch_dependent(k_resnorm_colsum, dim3((unsigned)(K / 32), a.post_gamma || a.gate ? 2u : 1u, 1), dim3(256), 0, st,
                            a, (const float*)ws, nblocks, K);
}

}  // namespace fp8rl
