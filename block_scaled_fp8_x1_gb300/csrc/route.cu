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
// One warp per row; lane l holds the NL neighbouring experts from l NL on, whose comparisons run on
// integers that order as the values do (0: cannot be selected), so a step of the selection is a
// scan of the lane's own values, a redux and a ballot.  The lowest lane, and in it the lowest place,
// is the lowest index.
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

// Keys of FP64 values: (hi, lo) order as the values do, 0 for -inf; NaN above all.
__device__ __forceinline__ uint64_t order_key64(double v) {
    if (v != v) return ~0ull;
    if (v == -INFINITY) return 0ull;
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ double key_value64(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}
__device__ __forceinline__ uint32_t reduce_max(uint32_t k) { return __reduce_max_sync(kFull, k); }
__device__ __forceinline__ uint64_t reduce_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint32_t key_sum(uint32_t a, uint32_t b) { return order_key(key_value(a) + key_value(b)); }
__device__ __forceinline__ uint64_t key_sum(uint64_t a, uint64_t b) { return order_key64(key_value64(a) + key_value64(b)); }

// Zeroes the keys of the experts outside the top_groups best groups.  Returns the ranks of the
// worst group kept and the best one left (0 if none is left).
template <int NL, typename KEY>
__device__ __forceinline__ void keep_groups(const fp8rl_route_args& a, int E, uint32_t gs_mul, int lane, KEY (&key)[NL], KEY* worst, KEY* left) {
    const int G = a.n_groups, gs = E / G;
    const int lpg = gs / NL;                            // lanes of a group
    KEY score = 0;                                      // lane g: rank of group g
    if (gs % NL == 0 && (lpg & (lpg - 1)) == 0) {
        // every group is lpg neighbouring lanes: its two best in log2(lpg) exchanges
        KEY b1 = 0, b2 = 0;
        #pragma unroll
        for (int i = 0; i < NL; ++i) {
            b2 = max(b2, min(b1, key[i]));
            b1 = max(b1, key[i]);
        }
        for (int o = 1; o < lpg; o <<= 1) {
            const KEY o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        if (a.group_rank == 2 && b2 != 0) b1 = key_sum(b1, b2);
        score = __shfl_sync(kFull, b1, (lane * lpg) & 31);
    } else {
        for (int g = 0; g < G; ++g) {
            KEY b1 = 0, b2 = 0;
            #pragma unroll
            for (int i = 0; i < NL; ++i) {
                const KEY k = group_of((uint32_t)(lane * NL + i), gs_mul) == (uint32_t)g ? key[i] : 0;
                b2 = max(b2, min(b1, k));
                b1 = max(b1, k);
            }
            KEY t = reduce_max(b1);
            if (a.group_rank == 2) {
                const uint32_t holder = __ballot_sync(kFull, b1 == t);
                const KEY second = reduce_max(lane == __ffs(holder) - 1 ? b2 : b1);
                if (second != 0) t = key_sum(t, second);
            }
            if (lane == g) score = t;
        }
    }
    int before = 0;
    for (int g = 0; g < G; ++g) {
        const KEY o = __shfl_sync(kFull, score, g);
        before += (o > score || (o == score && g < lane)) ? 1 : 0;
    }
    const bool kept = lane < G && before < a.top_groups;
    const uint32_t keep = __ballot_sync(kFull, kept);
    if (worst) {
        *worst = ~reduce_max(kept ? (KEY)~score : (KEY)0);
        *left = reduce_max(!kept && lane < G ? score : (KEY)0);
    }
    #pragma unroll
    for (int i = 0; i < NL; ++i)
        if (!((keep >> (group_of((uint32_t)(lane * NL + i), gs_mul) & 31u)) & 1u)) key[i] = 0;
}

// The largest key left, and its expert if there is one (0: none): the expert's key is zeroed.
template <int NL, typename KEY>
__device__ __forceinline__ KEY take_best(KEY (&key)[NL], int lane, int* expert) {
    KEY b = key[0];
    #pragma unroll
    for (int i = 1; i < NL; ++i) b = max(b, key[i]);
    const KEY top = reduce_max(b);
    if (top == 0) return 0;
    const int owner = __ffs(__ballot_sync(kFull, b == top)) - 1;
    int at = 0;
    #pragma unroll
    for (int i = NL - 1; i >= 0; --i)
        if (key[i] == top) at = i;
    #pragma unroll
    for (int i = 0; i < NL; ++i)
        if (lane == owner && i == at) key[i] = 0;
    *expert = __shfl_sync(kFull, lane * NL + at, owner);
    return top;
}

// The selection of one row from FP64 scores (rows with a near tie): lane j returns the j-th expert.
template <int NL, bool BF16>
__device__ __noinline__ int select_f64(const fp8rl_route_args& a, int64_t row, int E, uint32_t gs_mul, int lane) {
    const bool sm = a.score == FP8RL_SCORE_SOFTMAX;
    const int64_t base = row * a.ld;
    double v[NL];
    uint64_t key[NL];
    float m = -INFINITY;
    #pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane * NL + i;
        const float z = e < E ? load_logit<BF16>(a.logits, base + e) : -INFINITY;
        m = fmaxf(m, z);
        v[i] = (double)z;
        key[i] = z == -INFINITY ? 0ull : 1ull;      // 1: may be selected
    }
    m = warp_max(m);
    double sum = 0.0;
    #pragma unroll 1
    for (int i = 0; i < NL; ++i) {
        if (key[i]) v[i] = sm ? exp(v[i] - (double)m) : 1.0 / (1.0 + exp(-v[i]));
        if (key[i]) sum += v[i];
    }
    if (sm) sum = warp_sum(sum);
    #pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane * NL + i;
        double x = sm ? v[i] / sum : v[i];
        if (a.bias && e < E) x += (double)__ldg(a.bias + e);
        if (key[i]) key[i] = order_key64(x);
    }
    if (a.n_groups > 1) keep_groups<NL, uint64_t>(a, E, gs_mul, lane, key, nullptr, nullptr);
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        int e = 0;
        if (take_best<NL, uint64_t>(key, lane, &e) == 0) break;
        if (lane == j) mine = e;
    }
    return mine;
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
        const int e = lane * NL + i;
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
                if (lane * NL + i < E) t += expf(z[i] - m);
            inv = 1.0f / warp_sum(t);
        }
    }
    uint32_t key[NL];
    #pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane * NL + i;
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
        uint32_t worst, left;
        keep_groups<NL, uint32_t>(a, E, gs_mul, lane, key, &worst, &left);
        if (!by_logit && left != 0) {
            // sums of two: twice the error on each side, and their own rounding
            const float v = key_value(worst);
            close = !(v - key_value(left) > 6.0f * score_error(v, smax, sm));
        }
    }
    int mine = -1;              // lane j: the j-th expert
    uint32_t last = 0;
    for (int j = 0; j < a.k; ++j) {
        int e = 0;
        const uint32_t top = take_best<NL, uint32_t>(key, lane, &e);
        if (top == 0) break;
        if (lane == j) mine = e;
        if (j > 0 && !by_logit) {
            const float v = key_value(last);
            close = close || !(v - key_value(top) > 3.0f * score_error(v, smax, sm));
        }
        last = top;
    }
    if (!by_logit && last != 0) {
        // the best of those not taken (if any) against the last one taken
        uint32_t b = key[0];
        #pragma unroll
        for (int i = 1; i < NL; ++i) b = max(b, key[i]);
        b = __reduce_max_sync(kFull, b);
        const float v = key_value(last);
        close = close || (b != 0 && !(v - key_value(b) > 3.0f * score_error(v, smax, sm)));
    }
    if (close) mine = select_f64<NL, BF16>(a, row, E, gs_mul, lane);
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
