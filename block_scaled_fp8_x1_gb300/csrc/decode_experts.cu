// decode_experts.cu -- the experts' forward products for rollout: a few rows an expert, weights on
// the MMA's M side.
//
//     Y[r, n] = sum_kb sx(kb, r) sw_e(n / 128, kb) sum_{k in kb} X[r, k] W_e[n, k]
// for the rows r of each expert e, with the numerics of the other products.  The weights of the
// experts that have rows cross HBM once and bound the time, as in decode.cu, whose tile this is
// (A = 128 weight rows x 128, B = the activations of up to MP rows).
//
// Work: items (unit, weight tile), a unit being up to MP rows of one expert.  A CTA takes half of an
// SM's shared memory and registers.  Two CTAs an SM walk the items with one continuous copy / MMA /
// epilogue pipeline each: a CTA's start (about 5 us from launch to its first sums: the counts,
// tensor memory, the first copies) is paid once, not per item (61 tokens, 6 of 64 experts of 3584 x 1408:
// 58 us with an item a CTA, 52 this way).  Where the items are fewer than the SMs, a cluster of S CTAs
// shares each item's reduction instead and adds its FP32 sums in rank order through distributed shared
// memory.
// The host knows only how many units there can be; each CTA sums up the experts' units from the
// counts when it starts.
// Rows of a segment start anywhere: the copy of X has the rows of the next expert behind the
// unit's, which give columns that are not stored.
// Every mbarrier wait is bounded (FP8RL_ERR_DEVICE_TIMEOUT).
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "experts.h"

namespace fp8rl {

namespace {

constexpr int kThreads = 384;

template <int MP>
struct XDecodeCfg {
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int X_BYTES = MP * 128;
    static constexpr int STAGES = MP <= 32 ? 5 : 4;
    static constexpr int NB = 4;                     // TMEM buffers of MP columns
    static constexpr int COLS = NB * MP;             // TMEM columns, half of an SM's at most
    static constexpr int NSC = 8;                    // scale-ring slots
    static constexpr int SLOT = MP + 4;              // floats: the rows' scales, the weight block's
    static constexpr int CPT = MP / 2;               // columns (rows of X) per epilogue thread
    static constexpr int LW = CPT >= 32 ? 32 : 16;   // columns per TMEM load
    static constexpr size_t STAGE_BYTES = (size_t)STAGES * (W_BYTES + X_BYTES);
    static_assert((size_t)MP * 128 * 4 <= STAGE_BYTES, "the reduction buffer reuses the stage ring");
    static constexpr int NBARS = 2 * STAGES + 2 * NB + 3 * NSC + 1;
    static constexpr size_t FIXED = 1024 + STAGE_BYTES + (size_t)NSC * (SLOT + MP) * 4 + NBARS * 8 + 16 + 16 * 4;
    static size_t bytes(int E) { return FIXED + (2 * (size_t)E + 1) * 4; }
    static_assert(COLS <= 256 && FIXED + (2 * kMaxExperts + 1) * 4 <= 113 * 1024, "two CTAs an SM");
};

}  // namespace

template <int MP>
__global__ void __launch_bounds__(kThreads, 2)
    k_decode_experts(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                     const ExpertDecodeParams p) {
    using C = XDecodeCfg<MP>;
    constexpr int STAGES = C::STAGES, NB = C::NB, NSC = C::NSC, CPT = C::CPT, LW = C::LW, SLOT = C::SLOT;
    constexpr uint32_t IDESC = idesc_e4m3_f32(128, MP);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sW = smem;
    uint8_t* sX = smem + STAGES * C::W_BYTES;
    float* red = reinterpret_cast<float*>(smem);                               // after the last K-block
    float* sc_ring = reinterpret_cast<float*>(smem + C::STAGE_BYTES);          // [NSC][SLOT] copied scales
    float* comb = sc_ring + NSC * SLOT;                                        // [NSC][MP] combined scales
    uint64_t* bars = reinterpret_cast<uint64_t*>(comb + NSC * MP);
    uint64_t* full_bar = bars;                  // [STAGES] tile copies -> MMA
    uint64_t* empty_bar = bars + STAGES;        // [STAGES] MMA -> copies
    uint64_t* tfull_bar = bars + 2 * STAGES;    // [NB] MMA -> epilogue
    uint64_t* tempty_bar = tfull_bar + NB;      // [NB] epilogue -> MMA
    uint64_t* sfull_bar = tempty_bar + NB;      // [NSC] scale copies landed -> combiner
    uint64_t* cfull_bar = sfull_bar + NSC;      // [NSC] combined scales -> epilogue
    uint64_t* sempty_bar = cfull_bar + NSC;     // [NSC] epilogue -> scale copies
    uint64_t* drain_bar = sempty_bar + NSC;     // [1] MMA completion at exit
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_warp = reinterpret_cast<int*>(tmem_slot + 4);                       // [12] units of a warp's experts
    int* s_first = s_warp + 12;                                                // expert, first row and rows of this CTA's first unit
    int* s_units = s_warp + 16;                                                // [E + 1] units of the experts before
    int* s_start = s_units + p.E + 1;                                          // [E]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int S = (int)cluster_nctarank();
    const int rank = (int)cluster_ctarank();
    const int kb0 = (int)(((int64_t)rank * p.nkb) / S);
    const int kb1 = (int)(((int64_t)(rank + 1) * p.nkb) / S);
    const int nk = kb1 - kb0;                   // K-blocks of an item for this CTA (>= 1)

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int t = 0; t < NB; ++t) {
            mbar_init(smem_u32(&tfull_bar[t]), 1);
            mbar_init(smem_u32(&tempty_bar[t]), 8);
        }
        for (int t = 0; t < NSC; ++t) {
            mbar_init(smem_u32(&sfull_bar[t]), 32);   // one cp.async arrival per copy lane
            mbar_init(smem_u32(&cfull_bar[t]), 1);
            mbar_init(smem_u32(&sempty_bar[t]), 8);
        }
        mbar_init(smem_u32(drain_bar), 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::COLS);
        tmem_relinquish();
    }
    grid_dependency_begin();
    // units of the experts before each expert; the expert of the first unit is found on the way
    const int first = (int)cluster_idx(), step = (int)cluster_count();
    const int first_unit = (int)((uint32_t)first / (uint32_t)p.tiles);
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += kThreads) {
        const int e = e0 + (int)threadIdx.x;
        const int rows = e < p.E ? (int)min((int64_t)max(0, __ldg(p.count + e)), p.R) : 0, start = e < p.E ? __ldg(p.start + e) : 0;
        const int n = (rows + MP - 1) / MP;
        int scan = n;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) s_warp[warp] = scan;
        __syncthreads();
        int total = 0;
        #pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) scan += s_warp[i];
            total += s_warp[i];
        }
        if (e < p.E) {
            s_units[e] = carry + scan - n;
            s_start[e] = start;
            const int i = first_unit - (carry + scan - n);
            if (i >= 0 && i < n) {
                s_first[0] = e;
                s_first[1] = start + i * MP;
                s_first[2] = min(MP, rows - i * MP);
            }
        }
        carry += total;
        if (e0 + kThreads < p.E) __syncthreads();      // s_warp is written again
    }
    if (threadIdx.x == 0) s_units[p.E] = carry;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // items of this CTA: first, first + step, ... (one at most where the reduction is split), and no more
    // than the rows can have, whatever the counts
    const int items = (int)min((int64_t)max(carry, 0) * p.tiles, (int64_t)p.max_items);
    bool ok = true;
    // Item -> expert, weight tile and rows
    struct Item {
        int expert, tile, row0, rows;
    };
    auto item_at = [&](int item) {
        Item t;
        const int unit = (int)((uint32_t)item / (uint32_t)p.tiles);
        t.tile = item - unit * p.tiles;
        if (item == first) {
            t.expert = s_first[0];
            t.row0 = s_first[1];
            t.rows = s_first[2];
        } else {
            int e = 0, above = p.E;          // s_units[e] <= unit < s_units[above]
            while (above - e > 1) {
                const int mid = (e + above) >> 1;
                if (s_units[mid] <= unit) e = mid;
                else above = mid;
            }
            t.expert = e;
            const int before = (unit - s_units[e]) * MP;
            t.row0 = s_start[e] + before;
            t.rows = min(MP, max(0, __ldg(p.count + e)) - before);
        }
        // starts and counts that do not fit the rows: nothing is read or written there
        if (t.row0 < 0 || (int64_t)t.row0 + t.rows > p.R) {
            record_status(FP8RL_ERR_DEVICE_BOUNDS);
            t.row0 = t.rows = 0;
        }
        return t;
    };

    if (warp < 4) {
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            const uint64_t pol_w = l2_policy_evict_first();   // each weight byte is read once
            const uint64_t pol_x = l2_policy_evict_last();    // every tile reads the activation
            constexpr uint32_t TX = C::W_BYTES + C::X_BYTES;
            uint32_t it = 0;
            for (int item = first; ok && item < items; item += step) {
                const Item t = item_at(item);
                const int wy = (t.expert * p.tiles + t.tile) * 128;
                const float* swt = p.sw + ((int64_t)t.expert * p.tiles + t.tile) * p.nkb;
                for (int i = 0; i < nk; ++i, ++it) {
                    const int kb = kb0 + i;
                    const uint32_t s = it % STAGES;
                    if (!mbar_wait(smem_u32(&empty_bar[s]), ((it / STAGES) & 1) ^ 1, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (elect_one_sync()) {
                        mbar_arrive_expect_tx(smem_u32(&full_bar[s]), TX);
                        tma_load_2d(smem_u32(sW + s * C::W_BYTES), &tmW, smem_u32(&full_bar[s]), kb * 128, wy, pol_w);
                        tma_load_2d(smem_u32(sX + s * C::X_BYTES), &tmX, smem_u32(&full_bar[s]), kb * 128, t.row0, pol_x);
                    }
                    __syncwarp();
                    // this K-block's scales: sx(kb, r) of the unit's rows (zero behind them) and
                    // sw(tile, kb), by asynchronous copies whose landing completes the slot's barrier
                    const uint32_t ss = it % NSC;
                    if (!mbar_wait(smem_u32(&sempty_bar[ss]), ((it / NSC) & 1) ^ 1, p.timeout_ns, abort_flag)) {
                        ok = false;
                        ++it;
                        break;
                    }
                    const uint32_t slot = smem_u32(sc_ring + ss * SLOT);
                    const float* sxk = p.sx + (int64_t)kb * p.R + t.row0;
                    #pragma unroll
                    for (int c = lane; c < MP; c += 32) {
                        const bool v = c < t.rows;
                        cp_async_4(slot + 4u * (uint32_t)c, v ? sxk + c : p.sx, v ? 4u : 0u);
                    }
                    if (lane == 0) cp_async_4(slot + 4u * MP, swt + kb, 4u);
                    cp_async_arrive(smem_u32(&sfull_bar[ss]));
                }
            }
            // Drain: every issued copy lands before the stage memory is reused or freed.
            cp_async_wait_all();
            volatile int no_abort = 0;
            const uint32_t n_out = it < (uint32_t)STAGES ? it : (uint32_t)STAGES;
            for (uint32_t j = it - n_out; j < it; ++j)
                mbar_wait(smem_u32(&full_bar[j % STAGES]), (j / STAGES) & 1, p.timeout_ns, &no_abort);
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            const uint32_t w_base = smem_u32(sW), x_base = smem_u32(sX);
            uint32_t it = 0;
            for (int item = first; ok && item < items; item += step) {
                for (int i = 0; i < nk; ++i, ++it) {
                    const uint32_t ts = it % NB;
                    const uint32_t s = it % STAGES;
                    if (!mbar_wait(smem_u32(&tempty_bar[ts]), ((it / NB) & 1) ^ 1, p.timeout_ns, abort_flag) ||
                        !mbar_wait(smem_u32(&full_bar[s]), (it / STAGES) & 1, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + ts * MP;
                    const uint64_t da = sdesc_kmajor_sw128(w_base + s * C::W_BYTES);
                    const uint64_t db = sdesc_kmajor_sw128(x_base + s * C::X_BYTES);
                    if (elect_one_sync()) {
                        #pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32-byte steps inside the 128-byte rows
                            mma_f8(d, da + 2 * k, db + 2 * k, IDESC, k > 0 ? 1u : 0u);
                        mma_commit(smem_u32(&empty_bar[s]));
                        mma_commit(smem_u32(&tfull_bar[ts]));
                    }
                    __syncwarp();
                }
            }
            if (elect_one_sync()) mma_commit(smem_u32(drain_bar));
            __syncwarp();
            volatile int no_abort = 0;
            mbar_wait(smem_u32(drain_bar), 0, p.timeout_ns, &no_abort);
        } else if (warp == 2) {
            // ------------------------------------------------------------ scale combiner
            // per K-block, once for all epilogue threads: comb[r] = sx(kb, r) * sw(tile, kb)
            uint32_t it = 0;
            for (int item = first; ok && item < items; item += step) {
                for (int i = 0; i < nk; ++i, ++it) {
                    const uint32_t ss = it % NSC;
                    if (!mbar_wait(smem_u32(&sfull_bar[ss]), (it / NSC) & 1, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const float* src = sc_ring + ss * SLOT;
                    const float fw = src[MP];
                    #pragma unroll
                    for (int c = lane; c < MP; c += 32) comb[ss * MP + c] = src[c] * fw;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&cfull_bar[ss]));
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue warps
        const int quad = warp & 3;                    // TMEM lane quadrant of this warp
        const int col0 = ((warp - 4) >> 2) * CPT;     // first column (row of X) of this thread
        const int wrow = quad * 32 + lane;            // weight row within the tile
        const uint32_t tb_lane = tmem_base + ((uint32_t)(quad * 32) << 16) + col0;
        uint32_t it = 0;
        for (int item = first; ok && item < items; item += step) {
            float2 acc[CPT / 2];
            #pragma unroll
            for (int c = 0; c < CPT / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            for (int i = 0; i < nk; ++i, ++it) {
                const uint32_t ts = it % NB, ss = it % NSC;
                bool got = mbar_wait(smem_u32(&cfull_bar[ss]), (it / NSC) & 1, p.timeout_ns, abort_flag);
                got = got && mbar_wait(smem_u32(&tfull_bar[ts]), (it / NB) & 1, p.timeout_ns, abort_flag);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                tc_fence_after();
                const float* sc = comb + ss * MP + col0;
                uint32_t r[LW];
                static_assert(CPT == LW, "one TMEM load a K-block");
                tmem_ld_cols(tb_lane + ts * MP, r);
                tmem_ld_wait(r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&tempty_bar[ts]));
                #pragma unroll
                for (int j = 0; j < LW; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(sc + j);
                    acc[j / 2] = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                            make_float2(f.x, f.y), acc[j / 2]);
                    acc[j / 2 + 1] = __ffma2_rn(make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])),
                                                make_float2(f.z, f.w), acc[j / 2 + 1]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sempty_bar[ss]));
            }
            if (!ok) break;
            if (S == 1) {
                // the whole reduction is here: BF16 straight from registers, row by row (a warp's 32
                // weight rows of one token are 64 contiguous bytes)
                const Item t = item_at(item);
                uint16_t* yt = p.y + (int64_t)t.row0 * p.ldy + t.tile * 128 + wrow;
                #pragma unroll
                for (int c = 0; c < CPT / 2; ++c) {
                    const int t0 = col0 + 2 * c;
                    const uint32_t pk = pack_bf16x2(acc[c].x, acc[c].y);
                    if (t0 < t.rows) yt[(int64_t)t0 * p.ldy] = (uint16_t)(pk & 0xFFFFu);
                    if (t0 + 1 < t.rows) yt[(int64_t)(t0 + 1) * p.ldy] = (uint16_t)(pk >> 16);
                }
            } else {
                // every MMA of this CTA has completed and every tile copy was consumed by one, so the
                // stage ring is free: park this CTA's sums as red[row of X][weight row]
                #pragma unroll
                for (int c = 0; c < CPT / 2; ++c) {
                    red[(col0 + 2 * c) * 128 + wrow] = acc[c].x;
                    red[(col0 + 2 * c + 1) * 128 + wrow] = acc[c].y;
                }
            }
        }
    }

    // ---- cluster reduction: CTA r adds slice r of every CTA's partial sums in rank order
    __syncwarp();
    tc_fence_before();
    if (S > 1) {
        cluster_sync_all();
        if (warp >= 4 && *abort_flag == 0 && first < items) {
            const Item t = item_at(first);
            const int et = threadIdx.x - 128;                     // 0..255
            const int n4 = t.rows * 32;                           // float4s of the unit's rows
            const int per = (n4 + S - 1) / S;
            const int e_end = min(n4, (rank + 1) * per);
            const uint32_t red_local = smem_u32(red);
            for (int e = rank * per + et; e < e_end; e += 256) {
                const int tok = e >> 5;
                const int r4 = (e & 31) * 4;
                const uint32_t off = (uint32_t)(tok * 128 + r4) * 4u;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int j = 0; j < S; ++j) {
                    const float4 w = ld_dsmem_v4(mapa_shared(red_local + off, (uint32_t)j));
                    v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
                }
                uint2 o;
                o.x = pack_bf16x2(v.x, v.y);
                o.y = pack_bf16x2(v.z, v.w);
                *reinterpret_cast<uint2*>(p.y + (int64_t)(t.row0 + tok) * p.ldy + t.tile * 128 + r4) = o;
            }
        }
        cluster_sync_all();   // no CTA leaves while another still reads its shared memory
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::COLS);
    }
}

template <int MP>
static cudaError_t launch_t(const CUtensorMap& tw, const CUtensorMap& tx, const ExpertDecodeParams& p, int clusters,
                            int splits, cudaStream_t st) {
    auto kern = k_decode_experts<MP>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)XDecodeCfg<MP>::bytes((int)kMaxExperts));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * splits), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = XDecodeCfg<MP>::bytes(p.E);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)splits;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tw, tx, p);
}

int expert_decode_tokens(int64_t P, int64_t E) { return P <= 16 * std::min(P, E) ? 32 : 64; }

// CTAs that share an item's reduction: as many as leave no more CTAs than fit at once (two an SM),
// and at least 4 K-blocks each.  A second wave costs more than the split saves (88 tiles of 32
// K-blocks: one CTA each 14.2 us, 2 12.7, 3 12.4, 4 16.3, 8 20.2; 176 tiles: 19.0, 23.9, 22.7, 26.0, 34.3).
int expert_decode_splits(int64_t items, int64_t nkb, int num_sms) {
    int64_t s = 2 * (int64_t)num_sms / std::max<int64_t>(items, 1);
    s = std::min<int64_t>(s, nkb / 4);
    return (int)std::max<int64_t>(1, std::min<int64_t>(s, 8));
}

cudaError_t launch_decode_experts(const CUtensorMap& tw, const CUtensorMap& tx, const ExpertDecodeParams& p, int tokens,
                                  int clusters, int splits, cudaStream_t st) {
    return tokens == 32 ? launch_t<32>(tw, tx, p, clusters, splits, st) : launch_t<64>(tw, tx, p, clusters, splits, st);
}

// Reads and clears this translation unit's device status word.  The caller has synchronized the
// stream.
fp8rl_status read_and_clear_decode_experts_status() {
    unsigned int v = 0;
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof v) != cudaSuccess) return FP8RL_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_device_status, &zero, sizeof zero) != cudaSuccess) return FP8RL_ERR_CUDA;
    return static_cast<fp8rl_status>(v);
}

}  // namespace fp8rl
