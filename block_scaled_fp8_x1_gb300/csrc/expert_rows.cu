// expert_rows.cu -- between token order and expert order: the stable sort of (token, expert) pairs and
// the weighted sum back (the gather is in quantize.cu).
//
// Row layout (fp8rl_expert_layout): expert e's pairs, in the order of p = t k + j, take rows
// start[e] .. start[e] + count[e]; start[e + 1] is the next multiple of `align` after them.
#include <algorithm>

#include "common.cuh"
#include "experts.h"
#include "quant_common.cuh"

namespace fp8rl {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kSortWarps = 16;
constexpr int64_t kSortChunk = 2048;     // pairs of a block of the sort, at least
constexpr int kSortMaxBlocks = 128;

__device__ __forceinline__ uint4 ldg_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// ---------------------------------------------------------------- the sort

// Histogram of one block's pairs (an index outside [0, E) is no pair).
__global__ void __launch_bounds__(32 * kSortWarps) k_expert_hist(const int32_t* __restrict__ index, int64_t P, int E,
                                                                 int64_t chunk, int32_t* __restrict__ hist) {
    extern __shared__ int32_t s_hist[];
    grid_dependency_begin();
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * chunk, hi = min(lo + chunk, P);
    for (int64_t p = lo + threadIdx.x; p < hi; p += blockDim.x) {
        const int e = __ldg(index + p);
        if ((unsigned)e < (unsigned)E) atomicAdd(&s_hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(int64_t)blockIdx.x * E + e] = s_hist[e];
}

// Places one block's pairs.  Each warp has a contiguous part of them: the warps' counts, summed over
// the warps and blocks before, give every warp its first row of each expert, and within 32 pairs
// match_any ranks the pairs of one expert by lane, so the order is that of the pairs.
// s_n: [kSortWarps][E] counts, then first rows; s_start [E + 1]; s_count [E]; s_warp [kSortWarps].  All of it
// is the launch's own (place_smem): static arrays beside it would count towards the 48 KB that a launch has
// without asking.
constexpr size_t place_smem(int64_t E) { return ((size_t)(kSortWarps + 2) * E + 1 + kSortWarps) * 4; }
__global__ void __launch_bounds__(32 * kSortWarps) k_expert_place(const int32_t* __restrict__ index, int64_t P, int E,
                                                                  int64_t chunk, int align, int64_t R,
                                                                  const int32_t* __restrict__ hist, int32_t* __restrict__ pos,
                                                                  int32_t* __restrict__ src, int32_t* __restrict__ start,
                                                                  int32_t* __restrict__ count) {
    extern __shared__ int32_t s_n[];
    grid_dependency_begin();
    int32_t* const s_start = s_n + kSortWarps * E;
    int32_t* const s_count = s_start + E + 1;
    int32_t* const s_warp = s_count + E;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nb = gridDim.x, b = blockIdx.x;
    for (int i = tid; i < kSortWarps * E; i += blockDim.x) s_n[i] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)b * chunk, hi = min(lo + chunk, P);
    const int64_t part = ((hi - lo + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t wlo = min(lo + warp * part, hi), whi = min(wlo + part, hi);
    int32_t* const mine = s_n + warp * E;
    for (int64_t p = wlo + lane; p < whi; p += 32) {
        const int e = __ldg(index + p);
        if ((unsigned)e < (unsigned)E) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    // all pairs of expert e, those of the blocks before, and from the padded counts the starts
    int32_t carry = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + tid;
        int32_t all = 0, before = 0;
        if (e < E) {
            if (nb > 1) {
                #pragma unroll 8
                for (int i = 0; i < nb; ++i) {
                    const int32_t h = __ldg(hist + (int64_t)i * E + e);
                    all += h;
                    before += i < b ? h : 0;
                }
            } else {
                for (int w = 0; w < kSortWarps; ++w) all += s_n[w * E + e];
            }
        }
        const int32_t padded = (all + align - 1) / align * align;
        int32_t scan = padded;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(kFull, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) s_warp[warp] = scan;
        __syncthreads();
        int32_t off = carry, total = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            off += w < warp ? s_warp[w] : 0;
            total += s_warp[w];
        }
        if (e < E) {
            const int32_t first = off + scan - padded;
            s_start[e] = first;
            s_count[e] = all;
            int32_t at = first + before;
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t n = s_n[w * E + e];
                s_n[w * E + e] = at;
                at += n;
            }
        }
        carry += total;
        __syncthreads();
    }
    if (tid == 0) s_start[E] = carry;
    __syncthreads();
    if (b == 0) {
        for (int e = tid; e <= E; e += blockDim.x) start[e] = s_start[e];
        for (int e = tid; e < E; e += blockDim.x) count[e] = s_count[e];
    }
    for (int64_t p0 = wlo; p0 < whi; p0 += 32) {
        const int64_t p = p0 + lane;
        const int raw = p < whi ? __ldg(index + p) : -1;
        const int e = (unsigned)raw < (unsigned)E ? raw : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int32_t row = -1;
        if (e >= 0) row = mine[e] + rank;
        __syncwarp();
        if (e >= 0 && rank == 0) mine[e] += __popc(same);
        __syncwarp();
        if (p < whi) pos[p] = row;
        if (row >= 0) src[row] = (int32_t)p;
    }
    // rows of no pair: the experts' padding (a warp an expert) and the rest of the buffer
    if (align > 1)
        for (int e = b * kSortWarps + warp; e < E; e += nb * kSortWarps)
            for (int r = s_start[e] + s_count[e] + lane; r < s_start[e + 1]; r += 32) src[r] = -1;
    for (int64_t r = (int64_t)s_start[E] + (int64_t)b * blockDim.x + tid; r < R; r += (int64_t)nb * blockDim.x) src[r] = -1;
}

// ---------------------------------------------------------------- combine

// out[t] = residual[t] + sum_j weight[t, j] y[pos[t, j]] in FP32 in the order of j: a thread has 8
// columns of one token and the rows of up to SLOTS pairs (2, 4 or 8, by k) on their way at once.  Pairs without a row (pos
// outside [0, R)) add nothing.  A block has kCombine columns / 8 of one token (blockIdx.y: which), or
// with fewer columns several tokens.
constexpr int kCombine = 128;
template <int SLOTS>
__global__ void __launch_bounds__(kCombine) k_expert_combine(const uint16_t* __restrict__ y, int64_t ldy, int per,
                                                             const float* __restrict__ weight, const uint16_t* residual,
                                                             int64_t ldr, const int32_t* __restrict__ pos, int64_t T, int k,
                                                             int64_t R, uint16_t* out, int64_t ldo) {
    grid_dependency_begin();
    const int tokens = per < kCombine ? kCombine / per : 1;          // of a block
    const int mine = tokens > 1 ? (int)threadIdx.x / per : 0;
    const int chunk = tokens > 1 ? (int)threadIdx.x - mine * per : (int)(blockIdx.y * kCombine + threadIdx.x);
    const int64_t t = (int64_t)blockIdx.x * tokens + mine;
    if (mine >= tokens || t >= T || chunk >= per) return;
    const int64_t c = (int64_t)chunk * 8;
    uint4 res = make_uint4(0, 0, 0, 0);
    if (residual) res = *reinterpret_cast<const uint4*>(residual + t * ldr + c);
    float2 acc[4];
    #pragma unroll
    for (int h = 0; h < 4; ++h) acc[h] = make_float2(0.0f, 0.0f);
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
        int row[SLOTS];
        float w[SLOTS];
        #pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            row[j] = j0 + j < k ? __ldg(pos + t * k + j0 + j) : -1;
            w[j] = weight && j0 + j < k ? __ldg(weight + t * k + j0 + j) : 1.0f;
        }
        uint4 v[SLOTS];
        #pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const bool has = (unsigned)row[j] < (unsigned)R;
            v[j] = make_uint4(0, 0, 0, 0);
            if (has) v[j] = ldg_v4(y + (int64_t)row[j] * ldy + c);
            else w[j] = 0.0f;
        }
        #pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            #pragma unroll
            for (int h = 0; h < 4; ++h)
                acc[h] = __ffma2_rn(make_float2(w[j], w[j]), make_float2(bf16_lo(u[h]), bf16_hi(u[h])), acc[h]);
        }
    }
    const uint32_t u[4] = {res.x, res.y, res.z, res.w};
    uint32_t o[4];
    #pragma unroll
    for (int h = 0; h < 4; ++h) o[h] = pack_bf16x2(acc[h].x + bf16_lo(u[h]), acc[h].y + bf16_hi(u[h]));
    *reinterpret_cast<uint4*>(out + t * ldo + c) = make_uint4(o[0], o[1], o[2], o[3]);
}

// dweight[t, j] = <dout[t], y[pos[t, j]]>, a warp a pair; 0 for a pair without a row.
__global__ void __launch_bounds__(256) k_expert_dweight(const uint16_t* __restrict__ dout, int64_t ldd,
                                                        const uint16_t* __restrict__ y, int64_t ldy, int64_t N,
                                                        const int32_t* __restrict__ pos, int64_t P, int k, int64_t R,
                                                        float* __restrict__ dweight) {
    grid_dependency_begin();
    const int lane = threadIdx.x & 31;
    const int64_t p = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (p >= P) return;
    const int r = __ldg(pos + p);
    float acc = 0.0f;
    if ((unsigned)r < (unsigned)R) {
        const uint16_t* a = dout + (p / k) * ldd;
        const uint16_t* b = y + (int64_t)r * ldy;
        #pragma unroll 4
        for (int64_t c = lane * 8; c < N; c += 256) {
            const uint4 va = ldg_v4(a + c), vb = ldg_v4(b + c);
            const uint32_t ua[4] = {va.x, va.y, va.z, va.w}, ub[4] = {vb.x, vb.y, vb.z, vb.w};
            #pragma unroll
            for (int h = 0; h < 4; ++h) {
                acc = fmaf(bf16_lo(ua[h]), bf16_lo(ub[h]), acc);
                acc = fmaf(bf16_hi(ua[h]), bf16_hi(ub[h]), acc);
            }
        }
    }
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
    if (lane == 0) dweight[p] = acc;
}

}  // namespace

int expert_rows_blocks(int64_t P) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(kSortMaxBlocks, (P + kSortChunk - 1) / kSortChunk));
}

cudaError_t launch_expert_rows(const int32_t* index, int64_t P, int E, int align, int64_t R, int32_t* pos, int32_t* src,
                               int32_t* start, int32_t* count, int32_t* hist, cudaStream_t st) {
    const int nb = expert_rows_blocks(P);
    const int64_t chunk = (P + nb - 1) / nb;
    if (nb > 1) {
        const cudaError_t e = launch_dependent(k_expert_hist, dim3(nb), dim3(32 * kSortWarps), (size_t)E * 4, st, index, P, E, chunk, hist);
        if (e != cudaSuccess) return e;
    }
    const size_t smem = place_smem(E);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k_expert_place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)place_smem(kMaxExperts));
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(k_expert_place, dim3(nb), dim3(32 * kSortWarps), smem, st, index, P, E, chunk, align, R, hist, pos, src,
                            start, count);
}

cudaError_t launch_expert_combine(const uint16_t* y, int64_t ldy, int64_t N, const float* weight, const uint16_t* residual,
                                  int64_t ldr, const fp8rl_expert_layout& l, uint16_t* out, int64_t ldo, cudaStream_t st) {
    const int per = (int)(N / 8);
    const int tokens = per < kCombine ? kCombine / per : 1;
    const dim3 grid((unsigned)((l.T + tokens - 1) / tokens), (unsigned)(tokens > 1 ? 1 : (per + kCombine - 1) / kCombine));
    const auto kern = l.k <= 2 ? k_expert_combine<2> : l.k <= 4 ? k_expert_combine<4> : k_expert_combine<8>;
    return launch_dependent(kern, grid, dim3(kCombine), 0, st, y, ldy, per, weight, residual, ldr, l.pos, l.T, (int)l.k, l.R, out,
                            ldo);
}

cudaError_t launch_expert_dweight(const uint16_t* dout, int64_t ldd, const uint16_t* y, int64_t ldy, int64_t N,
                                  const fp8rl_expert_layout& l, float* dweight, cudaStream_t st) {
    const int64_t P = l.T * l.k;
    return launch_dependent(k_expert_dweight, dim3((unsigned)((P + 7) / 8)), dim3(256), 0, st, dout, ldd, y, ldy, N, l.pos, P,
                            (int)l.k, l.R, dweight);
}

}  // namespace fp8rl
