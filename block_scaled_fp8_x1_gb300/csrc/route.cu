// route.cu -- the router of an expert layer: scores of the experts, the k best of each token, their
// weights, and the gradient of the logits.
//
// For a row z of E logits:
//     s = softmax(z) or 1 / (1 + exp(-z)),   v = s + bias  (z itself without a bias and with group_rank 1),
//     the experts of the top_groups groups with the largest sums of their group_rank best v,
//     the k largest v among them, largest first, the lowest index first among equals,
//     weight_j = scale s_j / (sum_j s_j + 1e-20)  or  scale s_j.
//
// The selection is that of the scores themselves, to 2^-40 (sums with a bias: or 2^-44 of the largest of them): a
// token's experts do not change with the batch or with the last bits of an FP32 score.  Without a bias and with group_rank 1 the logits
// themselves are compared (both scores are increasing functions of them).  Otherwise the FP32 scores
// decide where they can (score_error), and where two neighbours of the order, or the groups' border,
// are too close for that, those few scores are formed again in pairs of FP32.
//
// One warp per row; lane l holds the NL neighbouring experts from l NL on, whose comparisons run on
// integers that order as the values do (0: cannot be selected).  The best keys are ranked by counting
// (sort_best); where that will not do, k steps of a scan of the lane's own values, a redux and a ballot
// (take_best).  The lowest lane, and in it the lowest place, is the lowest index.
#include "common.cuh"
#include "experts.h"

namespace fp8rl {

namespace {

constexpr int kRouteWarps = 4;          // rows of a block
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kTiny = 1e-20f;

// Integers in the order of the values: NaN (of either sign) above all, -0 as +0; 0 for -inf.
constexpr uint32_t kNegInf = 0x007fffffu;     // ~bits(-inf)
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);      // +0 for -0, and the positive NaN
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return max(k, kNegInf) - kNegInf;
}
__device__ __forceinline__ float key_value(uint32_t key) {
    const uint32_t k = key + kNegInf;
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

// The NL neighbours from e0 on of a row at p + base, -inf (or `none`) behind the last of E; in pieces of
// up to 16 bytes where `vec` says that rows are aligned to them (one number at a time touches every
// 32-byte sector of the row up to 8 times).
template <int NL, bool BF16>
__device__ __forceinline__ void load_lane(const void* p, int64_t base, int e0, int E, bool vec, float none, float (&z)[NL]) {
    constexpr int BYTES = NL * (BF16 ? 2 : 4);
    if (vec && e0 + NL <= E) {
        const char* at = reinterpret_cast<const char*>(p) + (base + e0) * (BF16 ? 2 : 4);
        uint32_t w[(BYTES + 3) / 4];
        if constexpr (BYTES >= 16) {
            #pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(at) + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else if constexpr (BYTES == 8) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
            w[0] = v.x; w[1] = v.y;
        } else if constexpr (BYTES == 4) {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
        } else {
            w[0] = __ldg(reinterpret_cast<const uint16_t*>(at));
        }
        #pragma unroll
        for (int i = 0; i < NL; ++i)
            z[i] = !BF16 ? __uint_as_float(w[i]) : (i & 1) ? __uint_as_float(w[i / 2] & 0xFFFF0000u) : __uint_as_float(w[i / 2] << 16);
        return;
    }
    #pragma unroll
    for (int i = 0; i < NL; ++i) z[i] = e0 + i < E ? load_logit<BF16>(p, base + e0 + i) : none;
}
// Whether rows of ld numbers from p on may be read so.
template <int NL, bool BF16>
bool lane_aligned(const void* p, int64_t ld) {
    constexpr int BYTES = NL * (BF16 ? 2 : 4), A = BYTES < 16 ? BYTES : 16;
    return reinterpret_cast<uintptr_t>(p) % A == 0 && ld * (BF16 ? 2 : 4) % A == 0;
}

__device__ __forceinline__ float sigmoid_f(float z) { return __frcp_rn(1.0f + expf(-z)); }
// s (1 - s) of the sigmoid s: even in z, e / (1 + e)^2 with e = exp(-|z|).  (1 - s from a rounded s loses its
// digits for large z: 1% at 12, all of them from 17 on.)
__device__ __forceinline__ float sigmoid_slope(float z) {
    const float e = expf(-fabsf(z)), r = __frcp_rn(1.0f + e);
    return e * r * r;
}

// Group of expert e, from mul = ceil(2^22 / group size): exact for e < 1024.
__device__ __forceinline__ uint32_t group_of(uint32_t e, uint32_t mul) { return (e * mul) >> 22; }

__device__ __forceinline__ uint32_t reduce_max(uint32_t k) { return __reduce_max_sync(kFull, k); }
__device__ __forceinline__ uint64_t reduce_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint32_t key_sum(uint32_t a, uint32_t b) { return order_key(key_value(a) + key_value(b)); }

// ---- scores in pairs of FP32 (hi + lo, |lo| <= half a unit of hi): Dekker's double-length arithmetic
// ("A floating-point technique for extending the available precision", Numer. Math. 18, 1971) with
// the products' errors by FMA.  A near tie settled in FP64 kept its warp, and with it the whole call,
// busy for 8 us: the FP64 unit is slow and the chains of an exponential and a division long.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair fast_two_sum(float a, float b) {        // |a| >= |b|
    const float s = __fadd_rn(a, b);
    return Pair{s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
    const Pair u = fast_two_sum(s.hi, __fadd_rn(s.lo, t.hi));
    return fast_two_sum(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    const float p = __fmul_rn(a.hi, b.hi);
    const float e = __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p)));
    return fast_two_sum(p, e);
}
__device__ __forceinline__ Pair operator/(Pair a, Pair b) {
    const float q = __fdiv_rn(a.hi, b.hi);
    const Pair r = a + Pair{-q, 0.0f} * b;
    const float q2 = __fdiv_rn(r.hi, b.hi);
    const Pair r2 = r + Pair{-q2, 0.0f} * b;
    const Pair s = fast_two_sum(q, q2);
    return fast_two_sum(s.hi, __fadd_rn(s.lo, __fdiv_rn(r2.hi, b.hi)));
}
// exp(x) for |x| <= 81, within 2^-41 of itself: x = n ln 2 + 8 t (Cody and Waite's reduction, ln 2 in
// three parts of which n times the first is exact), |t| <= 0.0434, the Taylor sum of t up to t^8 / 8!
// (the next term 2^-59; from t^4 on in FP32: 2^-23 of less than 2^-22), and three squarings.
__device__ __forceinline__ Pair exp_pair(Pair x) {
    const float n = rintf(__fmul_rn(x.hi, 1.44269504f));
    Pair r = Pair{x.hi, x.lo} + Pair{__fmul_rn(-n, 0x1.62e4p-1f), 0.0f};
    r = r + Pair{-n, 0.0f} * Pair{0x1.7f7d1cp-20f, 0x1.ef357ap-45f};
    const Pair t = Pair{r.hi * 0.125f, r.lo * 0.125f};
    const float h = t.hi, h2 = h * h;
    const float tail = h2 * h2 * (1.0f / 24 + h * (1.0f / 120 + h * (1.0f / 720 + h * (1.0f / 5040 + h * (1.0f / 40320)))));
    const Pair t2 = t * t;
    const Pair sixth = Pair{0x1.555556p-3f, -0x1.555556p-28f};       // 1 / 6
    Pair e = (t2 * t) * sixth + Pair{tail, 0.0f};
    e = Pair{0.5f * t2.hi, 0.5f * t2.lo} + e;
    e = Pair{1.0f, 0.0f} + (t + e);
    #pragma unroll
    for (int i = 0; i < 3; ++i) e = e * e;
    const float two_n = __int_as_float(((int)n + 127) << 23);
    return Pair{e.hi * two_n, e.lo * two_n};
}
__device__ __forceinline__ Pair shfl_xor(Pair v, int o) { return Pair{__shfl_xor_sync(kFull, v.hi, o), __shfl_xor_sync(kFull, v.lo, o)}; }

// Keys of pairs: hi, then lo; 0 for -inf, NaN above all.
__device__ __forceinline__ uint64_t order_key64(Pair v) {
    const uint32_t hi = order_key(v.hi);
    return hi == 0u ? 0ull : v.hi != v.hi ? ~0ull : ((uint64_t)hi << 32) | order_key(v.lo);
}
__device__ __forceinline__ Pair key_pair(uint64_t k) {
    if (k == ~0ull) return Pair{__int_as_float(0x7fffffff), 0.0f};
    return Pair{key_value((uint32_t)(k >> 32)), key_value((uint32_t)k)};
}

__device__ __forceinline__ uint64_t key_sum(uint64_t a, uint64_t b) { return order_key64(key_pair(a) + key_pair(b)); }

// The warp's largest of b1 over the lanes and, with rank 2, the next one (each lane holding its own two
// best; 0: none).
template <typename KEY>
__device__ __forceinline__ KEY two_best(KEY b1, KEY b2, int rank, int lane, KEY* second) {
    const KEY t = reduce_max(b1);
    *second = 0;
    if (rank == 2) {
        const uint32_t holder = __ballot_sync(kFull, b1 == t);
        *second = reduce_max(lane == __ffs(holder) - 1 ? b2 : b1);
    }
    return t;
}

// The larger magnitude of two keys' values.
__device__ __forceinline__ float key_size(uint32_t a, uint32_t b) { return fmaxf(fabsf(key_value(a)), fabsf(key_value(b))); }

// Lane g gets the rank of group g: the largest key of its experts, or the key of the two largest
// values' sum (0: no expert to select).  `addend`: the largest magnitude that a lane saw in such a sum.
template <int NL>
__device__ __forceinline__ uint32_t group_scores(const fp8rl_route_args& a, int E, uint32_t gs_mul, int lane, const uint32_t (&key)[NL],
                                                 float* addend) {
    using KEY = uint32_t;
    const int G = a.n_groups, gs = E / G;
    *addend = 0.0f;
    const int lpg = gs / NL;                            // lanes of a group
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
        if (a.group_rank == 2 && b2 != 0) {
            *addend = key_size(b1, b2);
            b1 = key_sum(b1, b2);
        }
        return __shfl_sync(kFull, b1, (lane * lpg) & 31);
    }
    KEY score = 0;
    for (int g = 0; g < G; ++g) {
        KEY b1 = 0, b2 = 0;
        #pragma unroll
        for (int i = 0; i < NL; ++i) {
            const KEY k = group_of((uint32_t)(lane * NL + i), gs_mul) == (uint32_t)g ? key[i] : 0;
            b2 = max(b2, min(b1, k));
            b1 = max(b1, k);
        }
        KEY second;
        KEY t = two_best(b1, b2, a.group_rank, lane, &second);
        if (second != 0) {
            *addend = fmaxf(*addend, key_size(t, second));
            t = key_sum(t, second);
        }
        if (lane == g) score = t;
    }
    return score;
}

// Which of the lanes with take set have the n largest keys, the lower lane first among equals.
template <typename KEY>
__device__ __forceinline__ uint32_t best_lanes(KEY key, bool take, int n, int lane) {
    int before = 0;
    for (uint32_t m = __ballot_sync(kFull, take); m; m &= m - 1) {
        const int g = __ffs(m) - 1;
        const KEY o = __shfl_sync(kFull, key, g);
        before += (o > key || (o == key && g < lane)) ? 1 : 0;
    }
    return __ballot_sync(kFull, take && before < n);
}

// Zeroes the keys of the experts of groups outside `keep`.
template <int NL, typename KEY>
__device__ __forceinline__ void keep_groups(uint32_t keep, int gs, uint32_t gs_mul, int lane, KEY (&key)[NL]) {
    if (gs % NL == 0) {                 // a lane's experts are of one group
        const bool in = (keep >> (group_of((uint32_t)(lane * NL), gs_mul) & 31u)) & 1u;
        #pragma unroll
        for (int i = 0; i < NL; ++i) key[i] = in ? key[i] : 0;
        return;
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

// Scores of a row in pairs.
template <bool BF16>
struct Fine {
    const fp8rl_route_args& a;
    int64_t base;
    float m;            // softmax: the row's maximum
    Pair sum;           // and the denominator
    __device__ __forceinline__ Pair power(float z) const {          // softmax: exp(z - m)
        const Pair d = two_sum(z, -m);
        if (!(d.hi > -80.0f)) return Pair{d.hi != d.hi ? d.hi : 0.0f, 0.0f};     // below 2^-115 of the sum
        return exp_pair(d);
    }
    __device__ __forceinline__ Pair score(float z) const {
        if (a.score == FP8RL_SCORE_SOFTMAX) return power(z) / sum;
        if (!(fabsf(z) <= 80.0f)) return Pair{z != z ? z : z > 0.0f ? 1.0f : 0.0f, 0.0f};   // within 2^-115
        return Pair{1.0f, 0.0f} / (Pair{1.0f, 0.0f} + exp_pair(Pair{-z, 0.0f}));
    }
    __device__ __forceinline__ uint64_t key(int e) const {          // 0: masked
        const float z = load_logit<BF16>(a.logits, base + e);
        if (z == -INFINITY) return 0;
        const Pair s = score(z);
        const float b = a.bias ? __ldg(a.bias + e) : 0.0f;
        return order_key64(fabsf(b) < INFINITY && s.hi == s.hi ? s + Pair{b, 0.0f} : Pair{s.hi + b, 0.0f});
    }
};
template <bool BF16>
__device__ __noinline__ Pair softmax_sum(const Fine<BF16>& x, int E, int lane) {
    Pair t = Pair{0.0f, 0.0f};
    for (int e = lane; e < E; e += 32) t = t + x.power(load_logit<BF16>(x.a.logits, x.base + e));
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t = t + shfl_xor(t, o);
    return t;
}
// The groups of `unsure` ranked by fine scores: which n of them are the best.
template <bool BF16>
__device__ __noinline__ uint32_t settle_groups(const Fine<BF16>& x, uint32_t unsure, int n, int gs, int lane) {
    uint64_t score = 0;
    for (uint32_t left = unsure; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        uint64_t b1 = 0, b2 = 0;
        for (int i = lane; i < gs; i += 32) {
            const uint64_t k = x.key(g * gs + i);
            b2 = max(b2, min(b1, k));
            b1 = max(b1, k);
        }
        uint64_t second;
        uint64_t t = two_best(b1, b2, x.a.group_rank, lane, &second);
        if (second != 0) t = key_sum(t, second);
        if (lane == g) score = t;
    }
    return best_lanes(score, (unsure >> lane) & 1u, n, lane);
}

// Lane j of the first n has an expert; returns the j-th of them by fine scores.
template <bool BF16>
__device__ __noinline__ int settle_order(const Fine<BF16>& x, int mine, int n, int lane) {
    const uint64_t key = mine >= 0 ? x.key(mine) : 0;
    int before = 0, got = -1;
    for (int j = 0; j < n; ++j) {
        const uint64_t o = __shfl_sync(kFull, key, j);
        const int e = __shfl_sync(kFull, mine, j);
        before += (o > key || (o == key && e < mine)) ? 1 : 0;
    }
    for (int j = 0; j < n; ++j) {
        const int r = __shfl_sync(kFull, before, j), e = __shfl_sync(kFull, mine, j);
        if (r == lane) got = e;
    }
    return got;
}

// The whole selection among the experts of the groups in `keep` from fine scores, for a row with
// more near ties than lanes.
template <int NL, bool BF16>
__device__ __noinline__ int select_fine(const Fine<BF16>& x, uint32_t keep, int E, uint32_t gs_mul, int lane) {
    uint64_t key[NL];
    #pragma unroll 1
    for (int i = 0; i < NL; ++i) key[i] = lane * NL + i < E ? x.key(lane * NL + i) : 0;
    keep_groups<NL, uint64_t>(keep, E / x.a.n_groups, gs_mul, lane, key);
    int mine = -1;
    for (int j = 0; j < x.a.k; ++j) {
        int e = 0;
        if (take_best<NL, uint64_t>(key, lane, &e) == 0) break;
        if (lane == j) mine = e;
    }
    return mine;
}

// The k + 1 largest keys at least, sorted: lane r gets the r-th (key, expert), the lowest expert first
// among equals, for r < the count returned; 0 where this way will not do (fewer lanes than k + 1 with
// a key, or more than 32 keys from the bound on).  The (k + 4)-th largest of the lanes' own maxima
// bounds the (k + 4)-th largest key from below, and few keys lie above it, so that a lane each holds
// them and ranks them by counting: a third of the instructions of k + 1 rounds of take_best.  (Four
// and not one, so that a near tie at the border seldom reaches past the keys that are sorted.)
template <int NL>
__device__ __forceinline__ int sort_best(const uint32_t (&key)[NL], int k, int lane, uint64_t* s_best, uint32_t* top, int* expert) {
    uint32_t b = key[0];
    #pragma unroll
    for (int i = 1; i < NL; ++i) b = max(b, key[i]);
    uint32_t bound = 0;
    for (int j = 0; j < k + 4; ++j) {
        const uint32_t t = __reduce_max_sync(kFull, b);
        if (t == 0 && j > k) break;
        bound = t;
        if (b == t) b = 0;
    }
    if (bound == 0) return 0;
    // the keys from the bound on, in the order of the experts: the lanes' counts summed up
    int mine = 0;
    #pragma unroll
    for (int i = 0; i < NL; ++i) mine += key[i] >= bound ? 1 : 0;
    int at = mine;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += v;
    }
    const int n = __shfl_sync(kFull, at, 31);
    if (n > 32) return 0;
    at -= mine;
    s_best[lane] = 0ull;
    __syncwarp();
    // (key, ~expert): greater first, the lowest expert first among equals
    #pragma unroll
    for (int i = 0; i < NL; ++i)
        if (key[i] >= bound) s_best[at++] = ((uint64_t)key[i] << 32) | (uint32_t)~(lane * NL + i);
    __syncwarp();
    const uint64_t own = s_best[lane];
    int before = 0;
    for (int j = 0; j < n; j += 4) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(s_best + j), v = *reinterpret_cast<const ulonglong2*>(s_best + j + 2);
        before += (u.x > own) + (u.y > own) + (v.x > own) + (v.y > own);
    }
    __syncwarp();
    if (lane < n) s_best[before] = own;
    __syncwarp();
    const uint64_t sorted = s_best[lane];
    *top = (uint32_t)(sorted >> 32);
    *expert = lane < n ? (int)~(uint32_t)sorted : -1;
    return n;
}

// Scores for the comparison, by the ex2.approx and rcp.approx instructions (each within 2^-22).
__device__ __forceinline__ float exp_quick(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmul_rn(x, 1.44269504f)));
    return r;
}
__device__ __forceinline__ float sigmoid_quick(float z) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp_quick(-z)));
    return r;
}
// How far an FP32 v may be from its value, the largest score of the row being smax.  exp_quick(x) is
// within 2^-22 + 2^-23 |x| of itself (its instruction; log2 e and the product round to 2^-24 each), so
// that a sigmoid, where |x| e^-|x| <= 0.37, is within 2^-20; a softmax within 2^-18, most of it the
// bound of its denominator's 36 additions in a row.  Adding the bias rounds by 2^-24 |v|.
__device__ __forceinline__ float score_error(float v, float smax, bool softmax) {
    return smax * (softmax ? 0x1p-18f : 0x1p-20f) + 0x1p-24f * fabsf(v);
}

// BY_LOGIT: neither a bias nor sums of two, the logits' order is the scores'.
template <int NL, bool BF16, bool BY_LOGIT>
__global__ void __launch_bounds__(32 * kRouteWarps) k_route(const fp8rl_route_args a, int64_t T, int E, uint32_t gs_mul, bool vec) {
    __shared__ __align__(16) uint64_t s_best[kRouteWarps][32];
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (row >= T) return;
    const int64_t base = row * a.ld;
    const bool sm = a.score == FP8RL_SCORE_SOFTMAX;
    constexpr bool by_logit = BY_LOGIT;
    float z[NL];
    load_lane<NL, BF16>(a.logits, base, lane * NL, E, vec, -INFINITY, z);
    float bias[NL];
    if (!BY_LOGIT && a.bias) load_lane<NL, false>(a.bias, 0, lane * NL, E, vec, 0.0f, bias);
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
            v = sm ? exp_quick(z[i] - m) * inv : sigmoid_quick(z[i]);
            if (a.bias) v += bias[i];
        }
        key[i] = order_key(v);
    }
    const float smax = sm ? inv : 1.0f;      // no score is larger
    Fine<BF16> fine{a, base, m, Pair{0.0f, 0.0f}};
    auto refine = [&] {
        if (sm && fine.sum.hi == 0.0f) fine.sum = softmax_sum<BF16>(fine, E, lane);
    };
    uint32_t keep = kFull;
    if (a.n_groups > 1) {
        float addend;
        const uint32_t score = group_scores<NL>(a, E, gs_mul, lane, key, &addend);
        keep = best_lanes(score, lane < a.n_groups, a.top_groups, lane);
        const bool kept = (keep >> lane) & 1u;
        const uint32_t worst = ~__reduce_max_sync(kFull, kept ? ~score : 0u);
        const uint32_t left = __reduce_max_sync(kFull, !kept && lane < a.n_groups ? score : 0u);
        if (!by_logit && left != 0) {
            // sums of two: twice the error on each side, and their own rounding; each of the two was rounded at
            // its own size, which with biases of both signs is more than the sum's (without a bias no more
            // than smax).  NaN and infinity let nothing pass.
            const float v = key_value(worst);
            float margin = 6.0f * score_error(v, smax, sm);
            if (a.bias && a.group_rank == 2) margin += 0x1.8p-22f * __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(addend)));
            if (!(v - key_value(left) > margin)) {
                // groups far enough above the best one left are in, those far below the worst kept out
                const float own = key_value(score);
                const bool in = kept && own - key_value(left) > margin, out = !kept && v - own > margin;
                const uint32_t unsure = __ballot_sync(kFull, lane < a.n_groups && score != 0 && !in && !out);
                const uint32_t sure = __ballot_sync(kFull, in);
                refine();
                keep = sure | settle_groups<BF16>(fine, unsure, a.top_groups - __popc(sure), E / a.n_groups, lane);
            }
        }
        keep_groups<NL, uint32_t>(keep, E / a.n_groups, gs_mul, lane, key);
    }
    int mine = -1;              // lane j: the j-th expert
    uint32_t top = 0;
    const int warp = threadIdx.x >> 5;
    const int n = NL > 1 ? sort_best<NL>(key, a.k, lane, s_best[warp], &top, &mine) : 0;
    if (n == 0) {
        for (int j = 0; j < a.k; ++j) {
            int e = 0;
            const uint32_t t = take_best<NL, uint32_t>(key, lane, &e);
            if (t == 0) break;
            if (lane == j) {
                mine = e;
                top = t;
            }
        }
    }
    if (!by_logit) {
        // neighbours of the order up to the first not taken that are too close, and how many of
        // those not taken may be as good as the last one taken
        const uint32_t next = __shfl_down_sync(kFull, top, 1);
        const uint32_t last = __shfl_sync(kFull, top, a.k - 1);
        const float v = key_value(top), vl = key_value(last), low = vl - 3.0f * score_error(vl, smax, sm);
        bool close = lane < a.k - (n == 0) && next != 0 && lane < 31 && !(v - key_value(next) > 3.0f * score_error(v, smax, sm));
        int more = __popc(__ballot_sync(kFull, lane >= a.k && lane < n && !(v < low)));
        bool whole = more > 0 && more == n - a.k;       // and those not sorted
        if (n == 0 && last != 0) {
            uint32_t b = key[0];
            #pragma unroll
            for (int i = 1; i < NL; ++i) b = max(b, key[i]);
            b = __reduce_max_sync(kFull, b);
            whole = b != 0 && !(key_value(b) < low);
        }
        close = __any_sync(kFull, close);
        if (close || more > 0 || whole) {
            refine();
            if (whole) mine = select_fine<NL, BF16>(fine, keep, E, gs_mul, lane);
            else mine = settle_order<BF16>(fine, mine, a.k + more, lane);
        }
    }
    if (lane >= a.k) mine = -1;
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
// where the last sum is c (sum_i g_i p_i / t) 1e-20 / t for renormalised weights: they change with the sum over
// all scores only as far as t is not far above the 1e-20.
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
    float s[NL];            // softmax: the scores; sigmoid: their derivatives
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
        for (int i = 0; i < NL; ++i) s[i] = sigmoid_slope(s[i]);
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
        // (above 1e-12 less than half a unit of the other terms: left out, so that experts that were not
        // chosen keep a gradient of 0)
        if (sm && t < 1e-12f) inner = mean * (kTiny / t);
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
        const float dz = s[i] * (d[i] - inner);      // sigmoid: inner is 0
        if (BF16) reinterpret_cast<uint16_t*>(a.dlogits)[row * a.ldd + e] = __bfloat16_as_ushort(__float2bfloat16_rn(dz));
        else reinterpret_cast<float*>(a.dlogits)[row * a.ldd + e] = dz;
    }
}

template <int NL>
cudaError_t route_t(const fp8rl_route_args& a, int64_t T, int E, cudaStream_t st) {
    const unsigned grid = (unsigned)((T + kRouteWarps - 1) / kRouteWarps);
    const uint32_t gs = (uint32_t)(E / a.n_groups);
    const uint32_t gs_mul = ((1u << 22) + gs - 1) / gs;
    const bool by_logit = a.bias == nullptr && (a.group_rank == 1 || a.n_groups == 1);
    const bool vec = (a.bf16 ? lane_aligned<NL, true>(a.logits, a.ld) : lane_aligned<NL, false>(a.logits, a.ld)) &&
                     lane_aligned<NL, false>(a.bias, 0);
    auto kern = a.bf16 ? (by_logit ? k_route<NL, true, true> : k_route<NL, true, false>)
                       : (by_logit ? k_route<NL, false, true> : k_route<NL, false, false>);
    kern<<<grid, 32 * kRouteWarps, 0, st>>>(a, T, E, gs_mul, vec);
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
