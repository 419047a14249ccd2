// route.cu -- the router of an expert layer: scores of the experts, the k best of each token, their
// weights, and the gradient of the logits.
//
// For a row z of E logits:
//     s = softmax(z) or 1 / (1 + exp(-z)),   v = s + bias  (z itself without a bias and with group_rank 1),
//     the experts of the top_groups groups with the largest sums of their group_rank best v,
//     the k largest v among them, largest first, the lowest index first among equals,
//     weight_j = scale s_j / (sum_j s_j + 1e-20)  or  scale s_j.
//
// Selection is exact: two runs, devices or batch sizes never disagree on an expert because of the
// last bits of a score.  Without a bias and with group_rank 1 the logits themselves are compared
// (both scores are increasing functions of them).  Otherwise the FP32 scores decide where they can
// (score_error), and a row in which two neighbours of the order, or the groups' border, are too
// close for that is decided again from FP64 scores.
//
// One warp per row; lane l holds experts l, l + 32, ..., whose comparisons run on integers that
// order as the values do (0: cannot be selected), so a step of the selection is two redux
// instructions and a scan of the lane's own values.
#include "common.cuh"
#include "experts.h"

namespace fp8rl {

namespace {

constexpr int kRouteWarps = 4;          // rows of a block
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kTiny = 1e-20f;

// Integers in the order of the values: NaN above all, -0 as +0; 0 for -inf.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xffffffffu;
    if (v == -INFINITY) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ float warp_max(float v) {
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if (BF16) return bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(p) + i));
    return __ldg(reinterpret_cast<const float*>(p) + i);
}

__device__ __forceinline__ float sigmoid_f(float z) { return __frcp_rn(1.0f + expf(-z)); }

// Group of expert e, from mul = ceil(2^22 / group size): exact for e < 1024.
__device__ __forceinline__ uint32_t group_of(uint32_t e, uint32_t mul) { return (e * mul) >> 22; }

// FP64 selection of one row (rows with a near tie).  order[j] of lane j: the j-th expert.
template <int NL, bool BF16>
__device__ __noinline__ int select_f64(const fp8rl_route_args& a, int64_t row, int E, int lane) {
    double v[NL];
    const bool sm = a.score == FP8RL_SCORE_SOFTMAX;
    const int64_t base = row * a.ld;
    float m = -INFINITY;
    for (int i = 0; i < NL; ++i) {
        const int e = i * 32 + lane;
        if (e < E) m = fmaxf(m, load_logit<BF16>(a.logits, base + e));
    }
    m = warp_max(m);
    double sum = 0.0;
    for (int i = 0; i < NL; ++i) {
        const int e = i * 32 + lane;
        const double z = e < E ? (double)load_logit<BF16>(a.logits, base + e) : -INFINITY;
        v[i] = sm ? exp(z - (double)m) : 1.0 / (1.0 + exp(-z));
        if (e < E) sum += v[i];
    }
    sum = warp_sum(sum);
    for (int i = 0; i < NL; ++i) {
        const int e = i * 32 + lane;
        if (sm) v[i] /= sum;
        if (e < E && a.bias) v[i] += (double)__ldg(a.bias + e);
        if (e >= E || load_logit<BF16>(a.logits, base + e) == -INFINITY) v[i] = -INFINITY;
        if (v[i] != v[i]) v[i] = INFINITY;      // NaN first
    }
    // the largest of the warp below or at (value, index) limits: lowest index among equals
    auto best = [&](double mine, int idx) {
        for (int o = 16; o >= 1; o >>= 1) {
            const double ov = __shfl_xor_sync(kFull, mine, o);
            const int oi = __shfl_xor_sync(kFull, idx, o);
            if (ov > mine || (ov == mine && oi < idx)) { mine = ov; idx = oi; }
        }
        return make_double2(mine, (double)idx);
    };
    if (a.n_groups > 1) {
        const int gs = E / a.n_groups;
        double score = -INFINITY;
        for (int g = 0; g < a.n_groups; ++g) {
            double tot = -INFINITY;
            int taken = -1;
            for (int r = 0; r < a.group_rank; ++r) {
                double mine = -INFINITY;
                int idx = 1 << 20;
                for (int i = 0; i < NL; ++i) {
                    const int e = i * 32 + lane;
                    if (e / gs == g && e != taken && v[i] > mine) { mine = v[i]; idx = e; }
                }
                const double2 b = best(mine, idx);
                if (b.x != -INFINITY) tot = tot == -INFINITY ? b.x : tot + b.x;
                taken = (int)b.y;
            }
            if (lane == g) score = tot;
        }
        int before = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const double o = __shfl_sync(kFull, score, g);
            before += (o > score || (o == score && g < lane)) ? 1 : 0;
        }
        const uint32_t keep = __ballot_sync(kFull, lane < a.n_groups && before < a.top_groups);
        for (int i = 0; i < NL; ++i) {
            const int e = i * 32 + lane;
            if (e < E && !((keep >> (e / gs)) & 1u)) v[i] = -INFINITY;
        }
    }
    int got = -1;
    for (int j = 0; j < a.k; ++j) {
        double mine = -INFINITY;
        int idx = 1 << 20;
        for (int i = 0; i < NL; ++i)
            if (v[i] > mine) { mine = v[i]; idx = i * 32 + lane; }
        const double2 b = best(mine, idx);
        const int e = (int)b.y;
        if (b.x == -INFINITY) break;
        if (lane == j) got = e;
        for (int i = 0; i < NL; ++i)
            if (i * 32 + lane == e) v[i] = -INFINITY;
    }
    return got;
}

// How far an FP32 v may be from its value, the largest score of the row being smax.  A sigmoid is
// within 2^-22 of itself (expf 1 ulp, a sum, a reciprocal); a softmax within 2^-18, nearly all of it
// the bound of its denominator's 36 additions in a row (rounding z - max adds at most
// x e^-x 2^-24 <= 2^-25).  Adding the bias rounds by 2^-24 |v|.
__device__ __forceinline__ float score_error(float v, float smax, bool softmax) {
    return smax * (softmax ? 0x1p-18f : 0x1p-22f) + 0x1p-24f * fabsf(v);
}

template <int NL, bool BF16>
__global__ void __launch_bounds__(32 * kRouteWarps) k_route(const fp8rl_route_args a, int64_t T, int E, uint32_t gs_mul) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (row >= T) return;
    const int64_t base = row * a.ld;
    const bool sm = a.score == FP8RL_SCORE_SOFTMAX;
    const bool by_logit = a.bias == nullptr && (a.group_rank == 1 || a.n_groups == 1);
    float z[NL];
    #pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * 32 + lane;
        z[i] = e < E ? load_logit<BF16>(a.logits, base + e) : -INFINITY;
    }
    // softmax: the row's maximum and sum, where something needs the scores of all experts
    float m = 0.0f, inv = 1.0f;
    if (sm) {
        m = z[0];
        #pragma unroll
        for (int i = 1; i < NL; ++i) m = fmaxf(m, z[i]);
        m = warp_max(m);
        if (!by_logit || !a.renormalize) {
            float t = 0.0f;
            #pragma unroll
            for (int i = 0; i < NL; ++i)
                if (i * 32 + lane < E) t += expf(z[i] - m);
            inv = 1.0f / warp_sum(t);
        }
    }
    uint32_t key[NL];
    #pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * 32 + lane;
        float v = z[i];
        if (!by_logit && e < E && z[i] != -INFINITY) {
            v = sm ? expf(z[i] - m) * inv : sigmoid_f(z[i]);
            if (a.bias) v += __ldg(a.bias + e);
        }
        key[i] = order_key(v);
    }
    const float smax = sm ? inv : 1.0f;      // no score is larger
    bool close = false;
    if (a.n_groups > 1) {
        // lane g keeps the score of group g; its experts' groups are e / (E / n_groups)
        uint32_t score = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            uint32_t b1 = 0, b2 = 0;
            #pragma unroll
            for (int i = 0; i < NL; ++i) {
                const uint32_t k = group_of((uint32_t)(i * 32 + lane), gs_mul) == (uint32_t)g ? key[i] : 0u;
                b2 = max(b2, min(b1, k));
                b1 = max(b1, k);
            }
            uint32_t s = __reduce_max_sync(kFull, b1);
            if (a.group_rank == 2) {
                const uint32_t holder = __ballot_sync(kFull, b1 == s);
                const uint32_t second = __reduce_max_sync(kFull, lane == __ffs(holder) - 1 ? b2 : b1);
                if (second != 0 && s != 0) s = order_key(key_value(s) + key_value(second));
            }
            if (lane == g) score = s;
        }
        int before = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const uint32_t o = __shfl_sync(kFull, score, g);
            before += (o > score || (o == score && g < lane)) ? 1 : 0;
        }
        const bool kept = lane < a.n_groups && before < a.top_groups;
        const uint32_t keep = __ballot_sync(kFull, kept);
        if (!by_logit) {
            const uint32_t lo = __reduce_min_sync(kFull, kept ? score : 0xffffffffu);
            const uint32_t hi = __reduce_max_sync(kFull, !kept && lane < a.n_groups ? score : 0u);
            if (hi != 0) {
                // sums of two: twice the error on each side, and their own rounding
                const float v = key_value(lo);
                close = !(v - key_value(hi) > 6.0f * score_error(v, smax, sm));
            }
        }
        #pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t g = group_of((uint32_t)(i * 32 + lane), gs_mul);
            if (!((keep >> (g & 31)) & 1u)) key[i] = 0;
        }
    }
    int mine = -1;              // lane j: the j-th expert
    uint32_t last = 0;
    for (int j = 0; j <= a.k; ++j) {
        uint32_t b = 0;
        #pragma unroll
        for (int i = 0; i < NL; ++i) b = max(b, key[i]);
        const uint32_t top = __reduce_max_sync(kFull, b);
        if (top == 0) break;
        if (j > 0 && !by_logit) {
            const float v = key_value(last);
            close = close || !(v - key_value(top) > 3.0f * score_error(v, smax, sm));
        }
        last = top;
        if (j == a.k) break;
        uint32_t idx = 0x7fffffffu;
        #pragma unroll
        for (int i = NL - 1; i >= 0; --i)
            if (key[i] == top) idx = i * 32 + lane;
        idx = __reduce_min_sync(kFull, idx);
        #pragma unroll
        for (int i = 0; i < NL; ++i)
            if ((uint32_t)(i * 32 + lane) == idx) key[i] = 0;
        if (lane == j) mine = (int)idx;
    }
    if (close) mine = select_f64<NL, BF16>(a, row, E, lane);
    float s = 0.0f;
    if (mine >= 0) {
        const float zz = load_logit<BF16>(a.logits, base + mine);
        s = sm ? expf(zz - m) * inv : sigmoid_f(zz);
    }
    float w = s;
    if (a.renormalize) w = s / (warp_sum(s) + kTiny);
    if (lane < a.k) {
        a.weight[row * a.k + lane] = mine >= 0 ? w * a.scale : 0.0f;
        a.index[row * a.k + lane] = mine;
    }
}

// dz from the gradient g of the weights: with c = scale, p the scores of the chosen experts and
// t = sum p + 1e-20,
//     ds_j = c g_j,  or renormalised  c (g_j - sum_i g_i p_i / t) / t,
//     sigmoid  dz_e = s_e (1 - s_e) ds_e,     softmax  dz_e = s_e (ds_e - sum_j ds_j p_j),
// where the last sum is 0 for renormalised weights (which do not change with the sum over all).
template <int NL, bool BF16>
__global__ void __launch_bounds__(32 * kRouteWarps) k_route_bwd(const fp8rl_route_bwd_args a, int64_t T, int E) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (row >= T) return;
    const int64_t base = row * a.ld;
    const bool sm = a.score == FP8RL_SCORE_SOFTMAX;
    int idx = -1;
    float g = 0.0f;
    if (lane < a.k) {
        idx = __ldg(a.index + row * a.k + lane);
        if (idx < 0 || idx >= E) idx = -1;
        if (idx >= 0) g = a.scale * __ldg(a.dweight + row * a.k + lane);
    }
    float s[NL];
    float m = -INFINITY;
    #pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * 32 + lane;
        s[i] = e < E ? load_logit<BF16>(a.logits, base + e) : -INFINITY;
        m = fmaxf(m, s[i]);
    }
    float inv = 1.0f;
    if (sm) {
        m = warp_max(m);
        float t = 0.0f;
        #pragma unroll
        for (int i = 0; i < NL; ++i) {
            s[i] = m == -INFINITY ? 0.0f : expf(s[i] - m);   // a row of masked experts has no scores
            t += s[i];
        }
        t = warp_sum(t);
        inv = t == 0.0f ? 0.0f : 1.0f / t;
        #pragma unroll
        for (int i = 0; i < NL; ++i) s[i] *= inv;
    } else {
        #pragma unroll
        for (int i = 0; i < NL; ++i) s[i] = sigmoid_f(s[i]);
    }
    float p = 0.0f;
    if (idx >= 0) {
        const float zz = load_logit<BF16>(a.logits, base + idx);
        p = !sm ? sigmoid_f(zz) : (m == -INFINITY ? 0.0f : expf(zz - m) * inv);
    }
    float inner = 0.0f;
    if (a.renormalize) {
        const float t = warp_sum(p) + kTiny;
        const float mean = warp_sum(g * p) / t;
        g = idx >= 0 ? (g - mean) / t : 0.0f;
    } else if (sm) {
        inner = warp_sum(g * p);
    }
    float d[NL];
    #pragma unroll
    for (int i = 0; i < NL; ++i) d[i] = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int e = __shfl_sync(kFull, idx, j);
        const float gj = __shfl_sync(kFull, g, j);
        #pragma unroll
        for (int i = 0; i < NL; ++i)
            if (i * 32 + lane == e) d[i] += gj;
    }
    #pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * 32 + lane;
        if (e >= E) continue;
        const float dz = sm ? s[i] * (d[i] - inner) : s[i] * (1.0f - s[i]) * d[i];
        if (BF16) reinterpret_cast<uint16_t*>(a.dlogits)[row * a.ldd + e] = __bfloat16_as_ushort(__float2bfloat16_rn(dz));
        else reinterpret_cast<float*>(a.dlogits)[row * a.ldd + e] = dz;
    }
}

template <int NL>
cudaError_t route_t(const fp8rl_route_args& a, int64_t T, int E, cudaStream_t st) {
    const unsigned grid = (unsigned)((T + kRouteWarps - 1) / kRouteWarps);
    const uint32_t gs = (uint32_t)(E / a.n_groups);
    const uint32_t gs_mul = ((1u << 22) + gs - 1) / gs;
    if (a.bf16) k_route<NL, true><<<grid, 32 * kRouteWarps, 0, st>>>(a, T, E, gs_mul);
    else k_route<NL, false><<<grid, 32 * kRouteWarps, 0, st>>>(a, T, E, gs_mul);
    return cudaGetLastError();
}

template <int NL>
cudaError_t route_bwd_t(const fp8rl_route_bwd_args& a, int64_t T, int E, cudaStream_t st) {
    const unsigned grid = (unsigned)((T + kRouteWarps - 1) / kRouteWarps);
    if (a.bf16) k_route_bwd<NL, true><<<grid, 32 * kRouteWarps, 0, st>>>(a, T, E);
    else k_route_bwd<NL, false><<<grid, 32 * kRouteWarps, 0, st>>>(a, T, E);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_topk(const fp8rl_route_args& a, int64_t T, int64_t E, cudaStream_t st) {
    if (E <= 32) return route_t<1>(a, T, (int)E, st);
    if (E <= 64) return route_t<2>(a, T, (int)E, st);
    if (E <= 128) return route_t<4>(a, T, (int)E, st);
    if (E <= 256) return route_t<8>(a, T, (int)E, st);
    if (E <= 512) return route_t<16>(a, T, (int)E, st);
    return route_t<32>(a, T, (int)E, st);
}

cudaError_t launch_route_topk_bwd(const fp8rl_route_bwd_args& a, int64_t T, int64_t E, cudaStream_t st) {
    if (E <= 32) return route_bwd_t<1>(a, T, (int)E, st);
    if (E <= 64) return route_bwd_t<2>(a, T, (int)E, st);
    if (E <= 128) return route_bwd_t<4>(a, T, (int)E, st);
    if (E <= 256) return route_bwd_t<8>(a, T, (int)E, st);
    if (E <= 512) return route_bwd_t<16>(a, T, (int)E, st);
    return route_bwd_t<32>(a, T, (int)E, st);
}

}  // namespace fp8rl
