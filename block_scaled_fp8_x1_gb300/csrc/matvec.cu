// matvec.cu -- y = x W^T for 1 to 16 tokens: BF16 activations on NVFP4 weights.
//
// "QeRL" (chatpaper.ai), abstract: rollout runs with NVFP4-quantized weights.  Here the weights
// alone are in 4 bits (nvfp4.cu gives the format and its layouts; the same q, sf, g serve its GEMM):
//     y[m][n] = bf16( g[n] sum_k x[m][k] e2m1(n,k) e4m3(n, k/16) ),
// with x as it is.
//
// Exactness.  e2m1 (2 significant bits) times e4m3 (4) has 6 and lies in 2^-10 .. 2688, so the
// weight w = e2m1 e4m3 is an FP16 number.  x goes to FP16 after a power-of-two scale for each token
// and 128 elements of K that takes their largest magnitude to [2^14, 2^15): its 8 significant bits
// fit, and only what is below 2^-28 of that maximum loses bits (an error below 2^-39 of it).  So
// the products are those of the given numbers and the FP16 tensor-core MMA sums them in FP32; the
// scale comes off in FP32, exactly.  There the row's g goes in as well, as far as it is a power of two
// (its fraction multiplies the finished sum): g is the row's largest weight / 2688, and sums in units
// of it would pass FP32's largest number where the result is 10^-4 of that.
//
// Work.  A unit is 32 weight rows x 128 of K: 2 KB of codes and 256 B of scales, which one warp
// copies to its own ring in shared memory (DEPTH units ahead) and multiplies with mma.m16n8k16:
// weights are the M side, up to 8 (or two times 8) tokens the N side.  The order of K inside the MMA is free as long
// as both operands agree: lane (g, t) = (lane / 4, lane % 4) takes the 16 bytes of K = 32t .. 32t+31
// of its rows, whose two scales sit in one 16-bit piece of the scale atom, and the matching x.  The
// rows of a unit are 8 o + g + 32 i (i = 0..3) of a 128-row group, so that one 16-byte load of the
// scale atom serves a lane's four rows.
//
// One token needs one column of the MMA's eight.  There the other columns separate the scale
// groups: the B operand holds lane t's x for its first (second) 16 of K in column 2t (2t + 1) and
// zero elsewhere, so column c of the product is the sum over scale group c of the 128 alone, of
// codes times x.  The scales then multiply 16 sums of a unit for a lane instead of its 128
// weights, and the columns are added at the end.
//
// Why mma.sync: tcgen05.mma takes the weights from shared or tensor memory, so each decoded weight
// would first be written there in 16 bits, four times its bytes from HBM, and read again.  From
// registers the same products cost 28 of the 98 cycles that HBM takes for a unit (up to 8 tokens).
//
// A CTA of 16 warps (one on an SM, so that x is laid out once for all of them) works on 16 / WK
// tiles of 32 rows at a time, WK warps splitting K, and a cluster
// of S CTAs splits K again; the parts are added in a fixed order (warps, then CTAs) through
// (distributed) shared memory.
//
// What bounds it.  One token on 37888 x 3584 (76 MB of weights): 17.2 us, 0.66 of the measured copy
// rate; reading the same pieces and doing nothing takes 14.4 us.  Eight tokens 20.8, sixteen 28.6 us:
// there the decoding (64 conversions and 64 multiplies a unit and lane, two of either a cycle an SM)
// and the 16 or 32 MMAs weigh more than the bytes.  Less than half of the issue slots are used in any of
// them: a unit is a chain of decoding, products and sums, and there are 16 warps.  3584 x 3584: 4.9 us,
// latency.
#include <cuda_fp16.h>

#include <algorithm>

#include "block.h"
#include "cluster.cuh"
#include "common.cuh"

namespace fp8rl {

namespace {

constexpr int kWarps = kMatvecWarps;
constexpr int kXBlock = 256;     // bytes of one token's 128 FP16 values in shared memory
constexpr int kUnit = 2304;      // bytes of a unit: 4 x 32 lanes x 16 of codes, 8 x 2 x 16 of scales

// Units that a warp has in flight, by the token slots (x takes the shared memory that is left).
__host__ __device__ constexpr int depth_of(bool one, int nt) { return one ? 5 : nt == 1 ? 3 : 2; }

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// Eight E2M1 codes -> four FP16 pairs (elements 2i, 2i+1 in h[i]), exactly.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into a fresh sum.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The power of two in a row scale, 2^-64 to 2^64, and its inverse: the sums run in units of what is
// left of the scale, so that they leave FP32's range only where the result does.
__device__ __forceinline__ uint32_t scale_exponent(float g) { return min(max(__float_as_uint(g) >> 23 & 255u, 63u), 191u); }
__device__ __forceinline__ float scale_power(float g) { return __uint_as_float(scale_exponent(g) << 23); }
__device__ __forceinline__ float scale_rest(float g) { return g * __uint_as_float((254u - scale_exponent(g)) << 23); }

struct Unit {
    uint4 w[4];   // codes of rows 8o + g + 32 i, K = 32t .. 32t + 31
    uint4 sf;     // their scale atom row: word i = row i's four scales of 64 elements
};

}  // namespace

// ONE: a single token (NT = 1); else NT groups of 8 tokens, a single one too where K is too long for
// the deeper ring of its own form.
template <bool ONE, int NT>
__global__ void __launch_bounds__(kWarps * 32, 1) k_matvec_nvfp4(const MatvecParams p) {
    grid_dependency_begin();
    extern __shared__ __align__(16) uint8_t mv_smem[];
    constexpr int TOK = ONE ? 1 : 8 * NT;                    // token slots of inv and red
    constexpr int DEPTH = depth_of(ONE, NT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int S = p.splits, WK = p.wk;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int ncl = (int)gridDim.x / S, cl = (int)blockIdx.x / S;
    const int nkb = p.nkb;                                   // K / 128
    const int kb0 = (int)((int64_t)nkb * rank / S), kb1 = (int)((int64_t)nkb * (rank + 1) / S);
    const int kslice = kb1 - kb0, kmax = (nkb + S - 1) / S;
    // the warps' rings; 16 zero bytes; x [kslice][M] blocks of kXBlock
    const uint32_t ring = smem_u32(mv_smem) + (uint32_t)(warp * DEPTH * kUnit);
    uint8_t* const zeros = mv_smem + kWarps * DEPTH * kUnit;
    uint8_t* xs = zeros + 16;
    float* inv = reinterpret_cast<float*>(xs + (size_t)kmax * p.M * kXBlock);   // [kslice][TOK]
    float* red = inv + (((size_t)kmax * TOK + 3) & ~(size_t)3);                 // [kWarps][TOK][32 rows]

    const int per = kWarps / WK;                             // tiles at a time
    const int ntile = p.tiles;                               // N / 32
    const int wt = warp / WK, wk = warp % WK;                // this warp's tile slot and K slot
    const int my_units = kslice > wk ? (kslice - wk + WK - 1) / WK : 0;
    // the warp's units in order, tile by tile; a copy past the last is an empty group
    int cp_tile = cl * per + wt, cp_un = 0, cp_slot = 0;
    auto copy_unit = [&]() {
        if (cp_tile < ntile && my_units > 0) {
            const int kb = kb0 + wk + cp_un * WK;
            const int64_t rg = cp_tile >> 2;
            const int o8 = 8 * (cp_tile & 3) + g;            // row within the atom's 32
            const uint8_t* w = p.qw + (rg * 128 + o8) * (int64_t)nkb * 64 + (int64_t)kb * 64 + 16 * t;
            const uint32_t dst = ring + (uint32_t)(cp_slot * kUnit);
            #pragma unroll
            for (int i = 0; i < 4; ++i) cp_async_16(dst + (uint32_t)(i * 512 + lane * 16), w + (int64_t)i * 32 * nkb * 64);
            if ((t & 1) == 0)                                // lanes 2a, 2a + 1 of a row share a scale atom
                cp_async_16(dst + 2048u + (uint32_t)(g * 32 + t * 8), p.sfw + (rg * nkb * 2 + 2 * kb + (t >> 1)) * 512 + o8 * 16);
            if (++cp_un == my_units) {
                cp_un = 0;
                cp_tile += ncl * per;
            }
        }
        cp_slot = cp_slot + 1 == DEPTH ? 0 : cp_slot + 1;
        cp_async_commit();
    };

    // the scales of this lane's four rows of the warp's next tile, requested a tile ahead
    float g_next[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    auto load_g = [&](int tile) {
        #pragma unroll
        for (int i = 0; i < 4; ++i)
            if (tile < ntile) g_next[i] = p.gw[(int64_t)(tile >> 2) * 128 + 32 * i + 8 * (tile & 3) + g];
    };
    load_g(cl * per + wt);

    // x to FP16 in fragment order: 16 lanes take one (K-block, token) block of 128.  Lane l holds
    // elements 8l .. 8l + 7, that is lane t = l / 4 of the MMA, quarter jj = l % 4: slot 4 jj + t.
    // The first loads go out before the first weights', the rest XB at a time.
    // (Odd tokens swap the slots' halves, so that two tokens of a load phase lie on other banks.)
    if (tid == 0) *reinterpret_cast<uint4*>(zeros) = make_uint4(0, 0, 0, 0);
    {
        constexpr int XB = ONE ? 2 : 6;
        const int l = tid & 15, items = kslice * p.M;
        uint4 xv[XB];
        auto load_x = [&](int it0) {
            #pragma unroll
            for (int q = 0; q < XB; ++q) {
                const int it = it0 + 2 * kWarps * q;
                const int kb = it / p.M, m = it - kb * p.M;
                xv[q] = make_uint4(0, 0, 0, 0);
                if (it < items) xv[q] = *reinterpret_cast<const uint4*>(p.x + (int64_t)m * p.ldx + (int64_t)(kb0 + kb) * 128 + 8 * l);
            }
        };
        load_x(tid >> 4);
        #pragma unroll
        for (int i = 0; i < DEPTH; ++i) copy_unit();
        for (int it0 = tid >> 4; it0 < items + (tid >> 4); it0 += 2 * kWarps * XB) {   // the same count in every warp
            #pragma unroll
            for (int q = 0; q < XB; ++q) {
                const int it = it0 + 2 * kWarps * q;
                if (it - (tid >> 4) >= items) break;   // the same in every thread
                const uint4 v = xv[q];
                uint32_t mx = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
                mx = max(mx & 0xFFFFu, mx >> 16);
                #pragma unroll
                for (int off = 8; off >= 1; off >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                // biased exponent of the maximum, at least 15 so that both factors are normal numbers
                const uint32_t e = max(mx >> 7, 15u);
                const float f = __uint_as_float((268u - e) << 23);          // 2^(141 - e)
                uint32_t h[4];
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t wv = word(v, j);
                    const float lo = __uint_as_float(wv << 16) * f, hi = __uint_as_float(wv & 0xFFFF0000u) * f;
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(hi), "f"(lo));
                }
                if (it < items) {
                    *reinterpret_cast<uint4*>(xs + (size_t)it * kXBlock + ((4 * (l & 3) + (l >> 2)) ^ (4 * (it % p.M & 1))) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
                    if (l == 0) inv[it / p.M * TOK + it % p.M] = __uint_as_float((e - 14u) << 23);   // 2^(e - 141)
                }
            }
            if (it0 + 2 * kWarps * XB < items + (tid >> 4)) load_x(it0 + 2 * kWarps * XB);
        }
    }
    __syncthreads();

    // this lane's column of each token group; columns past M repeat the last token and are not used
    uint32_t x_lane[NT], x_swap[NT];
    #pragma unroll
    for (int a = 0; a < NT; ++a) {
        const int m = 8 * a + g < p.M ? 8 * a + g : p.M - 1;
        x_lane[a] = smem_u32(xs) + (uint32_t)(m * kXBlock);
        x_swap[a] = 64u * (m & 1);
    }
    int slot = 0;
    for (int tile0 = cl * per; tile0 < ntile; tile0 += ncl * per) {
        const int tile = tile0 + wt;
        float gp[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) gp[i] = scale_power(g_next[i]);
        load_g(tile + ncl * per);
        float tot[NT][2][4];
        #pragma unroll
        for (int a = 0; a < NT; ++a)
            #pragma unroll
            for (int b = 0; b < 2; ++b)
                #pragma unroll
                for (int c = 0; c < 4; ++c) tot[a][b][c] = 0.0f;
        auto multiply = [&](const Unit& cur, int un) {
            const int kb = wk + un * WK;
            // scales of each row: groups 2t (K words 0, 1) and 2t + 1 (words 2, 3)
            uint32_t sc[4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint16_t pr = (uint16_t)(word(cur.sf, i) >> (16 * (t & 1)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(sc[i]) : "h"(pr));
            }
            float acc[NT][2][4];
            uint32_t s2[4][2];                               // !ONE: each group's scale in both halves
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                s2[i][0] = __byte_perm(sc[i], sc[i], 0x1010);
                s2[i][1] = __byte_perm(sc[i], sc[i], 0x3232);
            }
            #pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint4 b[NT];
                if (ONE) {
                    const uint8_t* at = g == 2 * t + (jj >> 1) ? xs + (size_t)kb * kXBlock + (4 * jj + t) * 16 : zeros;
                    b[0] = *reinterpret_cast<const uint4*>(at);
                } else {
                    #pragma unroll
                    for (int a = 0; a < NT; ++a)
                        b[a] = lds_v4(x_lane[a] + (uint32_t)(kb * p.M * kXBlock) + (((uint32_t)(64 * jj + 16 * t)) ^ x_swap[a]));
                }
                #pragma unroll
                for (int T = 0; T < 2; ++T) {
                    uint32_t ha[4], hb[4];
                    e2m1x8(word(cur.w[2 * T], jj), ha);
                    e2m1x8(word(cur.w[2 * T + 1], jj), hb);
                    if (!ONE) {
                        #pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            ha[i] = hmul2(ha[i], s2[2 * T][jj >> 1]);
                            hb[i] = hmul2(hb[i], s2[2 * T + 1][jj >> 1]);
                        }
                    }
                    #pragma unroll
                    for (int a = 0; a < NT; ++a) {
                        if (jj == 0) mma_f16_first(acc[a][T], ha[0], hb[0], ha[1], hb[1], b[a].x, b[a].y);
                        else mma_f16(acc[a][T], ha[0], hb[0], ha[1], hb[1], b[a].x, b[a].y);
                        mma_f16(acc[a][T], ha[2], hb[2], ha[3], hb[3], b[a].z, b[a].w);
                    }
                }
            }
            if (ONE) {
                // columns 2t, 2t + 1 are this lane's two scale groups
                const float iv = inv[kb];
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&sc[i]));
                    const float v = fmaf(acc[0][i >> 1][2 * (i & 1)], s.x, acc[0][i >> 1][2 * (i & 1) + 1] * s.y);
                    tot[0][0][i] = fmaf(v * gp[i], iv, tot[0][0][i]);
                }
            } else {
                #pragma unroll
                for (int a = 0; a < NT; ++a) {
                    const float2 iv = *reinterpret_cast<const float2*>(inv + kb * TOK + 8 * a + 2 * t);   // past M: unused
                    #pragma unroll
                    for (int T = 0; T < 2; ++T)
                        #pragma unroll
                        for (int i = 0; i < 2; ++i) {        // rows 2T and 2T + 1, columns 2t and 2t + 1
                            const float2 v = __fmul2_rn(make_float2(acc[a][T][2 * i], acc[a][T][2 * i + 1]), make_float2(gp[2 * T + i], gp[2 * T + i]));
                            const float2 s = __ffma2_rn(v, iv, make_float2(tot[a][T][2 * i], tot[a][T][2 * i + 1]));
                            tot[a][T][2 * i] = s.x;
                            tot[a][T][2 * i + 1] = s.y;
                        }
                }
            }
        };
        if (tile < ntile) {
            for (int un = 0; un < my_units; ++un) {
                cp_async_wait_group<DEPTH - 1>();
                __syncwarp();                                // the row's scales were copied by its even lanes
                const uint32_t src = ring + (uint32_t)(slot * kUnit);
                Unit cur;
                #pragma unroll
                for (int i = 0; i < 4; ++i) cur.w[i] = lds_v4(src + (uint32_t)(i * 512 + lane * 16));
                cur.sf = lds_v4(src + 2048u + (uint32_t)(g * 32 + (t >> 1) * 16));
                __syncwarp();                                // read by every lane: the slot takes the unit DEPTH ahead
                copy_unit();
                slot = slot + 1 == DEPTH ? 0 : slot + 1;
                multiply(cur, un);
            }
        }
        // parts to shared memory, [token][8 i + g] for row 8 o + g + 32 i
        if (ONE) {
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = tot[0][0][i];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (t == i) red[warp * 32 + 8 * i + g] = v;
            }
        } else {
            #pragma unroll
            for (int a = 0; a < NT; ++a)
                #pragma unroll
                for (int T = 0; T < 2; ++T)
                    #pragma unroll
                    for (int c = 0; c < 4; ++c)
                        red[(warp * TOK + 8 * a + 2 * t + (c & 1)) * 32 + 8 * (2 * T + (c >> 1)) + g] = tot[a][T][c];
        }
        __syncwarp();
        if (S > 1) cluster_sync_all();
        else __syncthreads();
        // outputs of the `per` tiles, shared out over the cluster: the parts in order
        const int n_out = per * p.M * 32;
        for (int i = rank * kWarps * 32 + tid; i < n_out; i += S * kWarps * 32) {
            const int r = i & 31, m = (i >> 5) % p.M, sl = (i >> 5) / p.M;
            const int tl = tile0 + sl;
            if (tl >= ntile) continue;
            float v = 0.0f;
            for (int s = 0; s < S; ++s) {
                const uint32_t at = smem_u32(red + ((sl * WK) * TOK + m) * 32 + r);
                const uint32_t from = S > 1 ? mapa_shared(at, (uint32_t)s) : at;
                for (int w = 0; w < WK; ++w) {
                    float q;
                    if (S > 1)
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q) : "r"(from + (uint32_t)w * TOK * 32 * 4) : "memory");
                    else
                        q = red[((sl * WK + w) * TOK + m) * 32 + r];
                    v += q;
                }
            }
            const int64_t n = (int64_t)(tl >> 2) * 128 + 32 * (r >> 3) + 8 * (tl & 3) + (r & 7);
            p.y[(int64_t)m * p.ldy + n] = (uint16_t)(pack_bf16x2(v * scale_rest(p.gw[n]), 0.0f) & 0xFFFFu);
        }
        // the next tiles' parts (or the exit of a CTA whose parts are still read)
        __syncwarp();
        if (S > 1) cluster_sync_all();
        else if (tile0 + ncl * per < ntile) __syncthreads();
    }
    cp_async_wait_all();
}

size_t matvec_smem(int M, int nkb, int splits, bool one) {
    const int tok = one ? 1 : (M + 7) / 8 * 8, kmax = (nkb + splits - 1) / splits;
    return (size_t)kWarps * depth_of(one, tok / 8) * kUnit + 16 + (size_t)kmax * M * kXBlock + (((size_t)kmax * tok + 3) & ~(size_t)3) * 4 + (size_t)kWarps * tok * 32 * 4;
}

cudaError_t launch_matvec_nvfp4(const MatvecParams& p, int clusters, cudaStream_t st) {
    const size_t smem = matvec_smem(p.M, p.nkb, p.splits, p.one);
    auto kern = p.one ? k_matvec_nvfp4<true, 1> : p.M <= 8 ? k_matvec_nvfp4<false, 1> : k_matvec_nvfp4<false, 2>;
    // one limit for every call: host threads may launch different sizes at once
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMatvecMaxSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(clusters * p.splits)), block(kWarps * 32);
    // clusters are launched plainly: set up ahead of the previous kernel's end they ran 2 us later
    // (3584 x 18944 at 11 tokens, clusters of 5: 21.1 against 18.9 us)
    if (p.splits == 1) return launch_dependent(kern, grid, block, smem, st, p);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace fp8rl
