// gemm_experts.cu -- block-scaled FP8 products of an expert layer on pairs of SMs (tcgen05
// cta_group::2): each expert's rows with its own weight matrix.
//
// With the rows in expert order, every expert's segment [start[e], start[e + 1]) a multiple of 128:
//   forward, DGrad   C[r, c] = sum_kb fa(kb, r) fb_e(kb, c / 128) sum_{k in kb} A[r, k] B_e[c, k]
//                    for the rows r of each expert e;
//   WGrad            C_e[n, k] = sum_kb fa(kb, n) fb(kb, k) sum_{r in kb} A[n, r] B[k, r]
//                    over the blocks kb of 128 rows of expert e (zeros where it has none);
// E4M3 x E4M3, FP32 sums of each 128-long block, promoted with the operands' scales into an FP32
// accumulator, BF16 results.
//
// One persistent launch for all experts: the pairs of SMs walk 256 x 256 result tiles in the order
// of the experts, so the tiles in flight share the rows and the weights of one or two experts
// through L2.  The segments are read on the device (the host does not know the counts): each CTA
// copies the E + 1 starts, and for forward and DGrad the running count of 256-row tiles, to shared
// memory.  A segment with an odd number of 128-row blocks leaves half of its last pair tile unused
// (computed on the next expert's rows, not stored).
//
// Roles and pipeline as in gemm_pair.cu: warp 2 finds the tiles and announces them to the others,
// warp 0 copies the operands, warp 3 the scales, warp 1 issues the MMAs, 8 (forward, DGrad) or 16
// (WGrad) epilogue warps promote each K-block's partial sums from one of two 256-column TMEM buffers.
// B's block scales (forward, DGrad) are read 32 K-blocks ahead, one a lane, and shuffled, so that any
// number of K-blocks and columns will do.
//
// What bounds it: the epilogue, which TMEM's two buffers keep in step with the MMAs.  Forward, 65536 rows
// of 64 experts: 0.40 us a K-block (0.35 without the promotion, 0.38 with it and no TMEM loads) and 1.8 us
// a tile; 580 us at 2816 x 4096, 2600 TFLOP/s.  WGrad: 0.56 us a K-block and 1.2 us for the tile's store,
// 840 us; without the promotion (a multiply and an FMA an element) 590.  The epilogue's registers are full (56
// bytes are spilled in the forward, 28 in WGrad): whatever adds a few more to its K loop costs more than it gives.
// Every mbarrier wait is bounded (FP8RL_ERR_DEVICE_TIMEOUT).
#include "common.cuh"
#include "experts.h"

namespace fp8rl {

namespace {

constexpr int kPN = 256;         // columns of a pair tile
constexpr int kBufs = 2;         // TMEM buffers of kPN columns

// Register split as in gemm_pair.cu.
__host__ __device__ constexpr int x_threads(int epi) { return 128 + 32 * epi; }
__host__ __device__ constexpr int x_launch_regs(int epi) { return epi == 16 ? 96 : 168; }
__host__ __device__ constexpr uint32_t x_reg_lo(int epi) { return epi == 16 ? 32 : 56; }
__host__ __device__ constexpr uint32_t x_reg_hi(int epi) { return epi == 16 ? 112 : 224; }
static_assert(128 * x_reg_lo(8) + 256 * x_reg_hi(8) <= x_threads(8) * x_launch_regs(8), "split");
static_assert(128 * x_reg_lo(16) + 512 * x_reg_hi(16) <= x_threads(16) * x_launch_regs(16), "split");

template <bool WGRAD>
struct XSmem {
    static constexpr int EPI = WGRAD ? 16 : 8;
    static constexpr int STAGES = 4;
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int B_BYTES = (kPN / 2) * 128;
    static constexpr int SG = WGRAD ? 1 : 4;              // K-blocks of a scale slot
    static constexpr int NS = WGRAD ? 8 : 4;              // scale slots
    static constexpr int SLOT_A = 128 * SG;               // floats
    static constexpr int SLOT = SLOT_A + (WGRAD ? kPN : 0);
    static constexpr int RING_BYTES = NS * SLOT * 4;
    static constexpr int STAGE_C_BYTES = 128 * kPN * 2;      // the whole result tile, 4 KB boxes
    static constexpr int NT = 4;                          // tiles announced ahead
    static constexpr int NBARS = 2 * STAGES + 2 * kBufs + 2 * NS + 2 * NT + 1;
    static size_t bytes(int E) {
        return 1024 + (size_t)STAGES * (A_BYTES + B_BYTES) + STAGE_C_BYTES + RING_BYTES + NBARS * 8 + 16 +
               NT * 32 + 2 * (size_t)(E + 1) * 4;
    }
};

// A tile of the result: expert, first row of this CTA's half, first column, K-blocks.
struct XTile {
    int e;
    int row;        // forward, DGrad: row of A and C; WGrad: row within the expert's result
    int row_end;    // end of the rows that are stored
    int col;
    int kb0;        // WGrad: first block of 128 rows
    int nkb;
};

// Walks item = first, first + step, ...; the experts only ever advance.
template <bool WGRAD>
struct XWalk {
    const int32_t* start;     // [E + 1]
    const int32_t* tiles;     // forward, DGrad: [E + 1] tiles of the experts before
    int E, n_tiles, rows, nkb;
    int e;                    // current expert
    __device__ __forceinline__ int total() const {
        return WGRAD ? E * ((rows + 255) / 256) * n_tiles : tiles[E];
    }
    __device__ __forceinline__ XTile at(int item, int rank) {
        XTile t;
        int m, n, units;
        if (WGRAD) {
            units = (rows + 255) / 256;
            e = item / (units * n_tiles);
            item -= e * units * n_tiles;
        } else {
            if (tiles[e + 1] <= item) {      // tiles[e] <= item < tiles[above]
                int above = E;
                while (above - e > 1) {
                    const int mid = (e + above) >> 1;
                    if (tiles[mid] <= item) e = mid;
                    else above = mid;
                }
            }
            item -= tiles[e];
            units = (start[e + 1] - start[e] + 255) / 256;
        }
        // within an expert 16 row units at a time sweep the columns, which keeps their rows (16 MB
        // at 4096 columns) and the expert's weights in L2
        raster_tile(item, units, n_tiles, 16, 0, &m, &n);
        t.e = e;
        t.col = n * kPN;
        if (WGRAD) {
            t.row = m * 256 + rank * 128;
            t.row_end = rows;
            t.kb0 = start[e] >> 7;
            t.nkb = max(0, start[e + 1] - start[e]) >> 7;
        } else {
            t.row = start[e] + m * 256 + rank * 128;
            t.row_end = start[e + 1];
            t.kb0 = 0;
            t.nkb = nkb;
        }
        return t;
    }
};

template <bool WGRAD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(x_threads(XSmem<WGRAD>::EPI), 1)
    k_gemm_experts(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                   const __grid_constant__ CUtensorMap tmC, const ExpertGemmParams p) {
    using S = XSmem<WGRAD>;
    constexpr int EPI = S::EPI, NS = S::NS, kStages = S::STAGES;
    constexpr int COLS = kPN / (EPI / 4);           // columns per epilogue thread
    constexpr uint32_t TMEM_COLS = 512;
    constexpr uint32_t IDESC = idesc_e4m3_f32(256, kPN);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kStages * S::A_BYTES;
    uint8_t* stage_c = sB + kStages * S::B_BYTES;                         // [warp][box][4 KB]
    float* ring = reinterpret_cast<float*>(stage_c + S::STAGE_C_BYTES);   // [NS][SLOT]
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ring) + S::RING_BYTES);
    uint64_t* full_bar = bars;                       // [stages] copies of both CTAs -> MMA (leader's)
    uint64_t* empty_bar = bars + kStages;            // [stages] MMA -> copies (each CTA's own)
    uint64_t* tfull_bar = bars + 2 * kStages;        // [bufs] MMA -> epilogue (each CTA's own)
    uint64_t* tempty_bar = tfull_bar + kBufs;        // [bufs] both epilogues -> MMA (leader's)
    uint64_t* sfull_bar = tempty_bar + kBufs;        // [NS] scale copies -> epilogue
    uint64_t* sempty_bar = sfull_bar + NS;           // [NS] epilogue -> scale copies
    uint64_t* dfull_bar = sempty_bar + NS;           // [NT] a tile announced -> all roles
    uint64_t* dempty_bar = dfull_bar + S::NT;        // [NT] all roles have it -> the next
    uint64_t* drain_bar = dempty_bar + S::NT;        // [1] MMA completion at exit (leader)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* s_tile = reinterpret_cast<int32_t*>(tmem_slot + 2);          // [NT][8], 16-byte aligned
    static_assert(S::NBARS % 2 == 1 && S::RING_BYTES % 16 == 0, "alignment of the announced tiles");
    int32_t* s_start = s_tile + S::NT * 8;                                // [E + 1]
    int32_t* s_tiles = s_start + p.E + 1;                                 // [E + 1]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    uint32_t cid, ncl;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(cid));
    asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(ncl));
    const int n_tiles = (p.cols + kPN - 1) / kPN;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int t = 0; t < kBufs; ++t) {
            mbar_init(smem_u32(&tfull_bar[t]), 1);
            mbar_init(smem_u32(&tempty_bar[t]), 2 * EPI);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&sfull_bar[s]), 1);
            mbar_init(smem_u32(&sempty_bar[s]), EPI);
        }
        for (int s = 0; s < S::NT; ++s) {
            mbar_init(smem_u32(&dfull_bar[s]), 1);
            mbar_init(smem_u32(&dempty_bar[s]), EPI + 2 + (leader ? 1 : 0));   // epilogue, copies, scales, MMA
        }
        mbar_init(smem_u32(drain_bar), 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSA);
        if (WGRAD) tma_prefetch_desc(&tmSB);
        tma_prefetch_desc(&tmC);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    grid_dependency_begin();
    if (warp == 2) {
        // the starts, and the experts' tiles by a running sum over 32 experts at a time
        int32_t carry = 0, last = 0;
        for (int e0 = 0; e0 <= p.E; e0 += 32) {
            const int e = e0 + lane;
            // within [0, R], aligned and ascending whatever the array holds: a copy has to start on 16
            // bytes, and the tiles have to stay as many as R rows can have
            auto at = [&](int i) { return min(max(__ldg(p.start + min(i, p.E)), 0), p.R) & ~127; };
            int32_t a = max(last, at(e));
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) a = max(a, __shfl_up_sync(0xffffffffu, a, o));
            const int32_t b = max(a, at(e + 1));
            last = __shfl_sync(0xffffffffu, a, 31);
            const int32_t n = e < p.E ? ((b - a + 255) / 256) * n_tiles : 0;
            int32_t scan = n;
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, scan, o);
                if (lane >= o) scan += v;
            }
            if (e <= p.E) {
                s_start[e] = a;
                s_tiles[e] = carry + scan - n;
            }
            carry += __shfl_sync(0xffffffffu, scan, 31);
        }
    }
    tc_fence_before();
    cluster_sync_all();   // both CTAs' barriers initialised, TMEM allocated, starts in place
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    XWalk<WGRAD> walk{s_start, s_tiles, p.E, n_tiles, p.rows, p.nkb, 0};
    const int num_items = walk.total();
    // This CTA's n-th tile, from the warp that works them out: every role waits for it once, reads it
    // and gives its place back.
    auto announced = [&](uint32_t n) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(&dfull_bar[n % S::NT]), (n / S::NT) & 1, p.timeout_ns, abort_flag));
    };
    auto told = [&](uint32_t n) {
        const int4* d = reinterpret_cast<const int4*>(s_tile + (n % S::NT) * 8);
        const int4 a = d[0], b = d[1];
        return XTile{a.x, a.y, a.z, a.w, b.x, b.y};
    };
    auto taken = [&](uint32_t n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&dempty_bar[n % S::NT]));
    };

    if (warp < 4) {
        warpgroup_reg_dealloc<x_reg_lo(EPI)>();
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            const uint64_t pol = l2_policy_evict_last();
            const uint32_t full0 = mapa_shared(smem_u32(full_bar), 0);   // the leader's
            uint32_t it = 0, nt = 0;
            bool ok = true;
            for (int item = (int)cid; ok && item < num_items; item += (int)ncl) {
                ok = announced(nt);
                if (!ok) break;
                const XTile t = told(nt);
                taken(nt++);
                const int ax = WGRAD ? t.kb0 * 128 : 0;                       // first reduction column of A
                const int bx = WGRAD ? t.kb0 * 128 : t.e * p.b_x;             // and of B
                const int by = (WGRAD ? 0 : t.e * p.b_y) + t.col + (int)rank * (kPN / 2);
                for (int kb = 0; kb < t.nkb; ++kb, ++it) {
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(smem_u32(&empty_bar[s]), ((it / kStages) & 1) ^ 1, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (elect_one_sync()) {
                        if (leader) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), 2 * (S::A_BYTES + S::B_BYTES));
                        tma_load_2d_pair(smem_u32(sA + s * S::A_BYTES), &tmA, full0 + 8 * s, ax + kb * 128, t.row, pol);
                        tma_load_2d_pair(smem_u32(sB + s * S::B_BYTES), &tmB, full0 + 8 * s, bx + kb * 128, by, pol);
                    }
                    __syncwarp();
                }
            }
            // Drain: the copies issued here land before the CTA can exit.
            volatile int no_abort = 0;
            if (leader) {
                const uint32_t n_out = it < (uint32_t)kStages ? it : (uint32_t)kStages;
                for (uint32_t j = it - n_out; j < it; ++j)
                    mbar_wait(smem_u32(&full_bar[j % kStages]), (j / kStages) & 1, p.timeout_ns, &no_abort);
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ tiles
            // worked out here, ahead of the others: finding it by themselves cost the epilogue warps 0.6 us
            // a tile, and six registers of the K loop
            uint32_t nt = 0;
            for (int item = (int)cid; item < num_items; item += (int)ncl, ++nt) {
                const XTile t = walk.at(item, (int)rank);
                const uint32_t d = nt % S::NT;
                if (!mbar_wait(smem_u32(&dempty_bar[d]), ((nt / S::NT) & 1) ^ 1, p.timeout_ns, abort_flag)) break;
                if (lane == 0) {
                    *reinterpret_cast<int4*>(s_tile + d * 8) = make_int4(t.e, t.row, t.row_end, t.col);
                    *reinterpret_cast<int4*>(s_tile + d * 8 + 4) = make_int4(t.kb0, t.nkb, 0, 0);
                    mbar_arrive(smem_u32(&dfull_bar[d]));
                }
                __syncwarp();
            }
        } else if (warp == 3) {
            // ------------------------------------------------------------ scales
            // a warp of their own, so that they run ahead by the whole scale ring (16 K-blocks, WGrad 8) and
            // not by the operands' 4 stages (B's block scales in forward and DGrad: the epilogue reads them)
            const uint64_t pol = l2_policy_evict_last();
            const int sgrp = WGRAD ? 1 : (p.nkb < S::SG ? p.nkb : S::SG);
            uint32_t it = 0, nt = 0;
            bool ok = true;
            for (int item = (int)cid; ok && item < num_items; item += (int)ncl) {
                ok = announced(nt);
                if (!ok) break;
                const XTile t = told(nt);
                taken(nt++);
                for (int kb = 0; kb < t.nkb; kb += S::SG, ++it) {
                    const uint32_t ss = it % NS;
                    if (!mbar_wait(smem_u32(&sempty_bar[ss]), ((it / NS) & 1) ^ 1, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sb = smem_u32(&sfull_bar[ss]);
                    float* slot = ring + ss * S::SLOT;
                    if (elect_one_sync()) {
                        mbar_arrive_expect_tx(sb, 128u * 4u * (uint32_t)sgrp + (WGRAD ? (uint32_t)kPN * 4u : 0u));
                        tma_load_2d(smem_u32(slot), &tmSA, sb, t.row, t.kb0 + kb, pol);
                        if (WGRAD) tma_load_2d(smem_u32(slot + S::SLOT_A), &tmSB, sb, t.col, t.kb0 + kb, pol);
                    }
                    __syncwarp();
                }
            }
            volatile int no_abort = 0;
            const uint32_t n_out = it < (uint32_t)NS ? it : (uint32_t)NS;
            for (uint32_t j = it - n_out; j < it; ++j)
                mbar_wait(smem_u32(&sfull_bar[j % NS]), (j / NS) & 1, p.timeout_ns, &no_abort);
        } else if (warp == 1 && leader) {
            // ------------------------------------------------------------ MMA issuer
            uint32_t it = 0, nt = 0;
            bool ok = true;
            const uint32_t a_base = smem_u32(sA), b_base = smem_u32(sB);
            for (int item = (int)cid; ok && item < num_items; item += (int)ncl) {
                ok = announced(nt);
                if (!ok) break;
                const XTile t = told(nt);
                taken(nt++);
                const int nkb = t.nkb;
                for (int kb = 0; kb < nkb; ++kb, ++it) {
                    const uint32_t ts = it % kBufs;
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(smem_u32(&tempty_bar[ts]), ((it / kBufs) & 1) ^ 1, p.timeout_ns, abort_flag) ||
                        !mbar_wait(smem_u32(&full_bar[s]), (it / kStages) & 1, p.timeout_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + ts * kPN;
                    const uint64_t da = sdesc_kmajor_sw128(a_base + s * S::A_BYTES);
                    const uint64_t db = sdesc_kmajor_sw128(b_base + s * S::B_BYTES);
                    if (elect_one_sync()) {
                        #pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32-byte steps inside the 128-byte rows
                            mma_f8_pair(d, da + 2 * k, db + 2 * k, IDESC, k > 0 ? 1u : 0u);
                        mma_commit_pair(smem_u32(&empty_bar[s]), 0x3);
                        mma_commit_pair(smem_u32(&tfull_bar[ts]), 0x3);
                    }
                    __syncwarp();
                }
            }
            // every MMA of the pair completes before either CTA frees its TMEM
            if (elect_one_sync()) mma_commit_pair(smem_u32(drain_bar), 0x1);
            __syncwarp();
            volatile int no_abort = 0;
            mbar_wait(smem_u32(drain_bar), 0, p.timeout_ns, &no_abort);
        }
    } else {
        warpgroup_reg_alloc<x_reg_hi(EPI)>();
        // ------------------------------------------------------------ epilogue warps
        const int ew = warp - 4;                 // 0 .. EPI-1
        const int quad = warp & 3;               // TMEM lane quadrant this warp may access
        const int col_base = (ew >> 2) * COLS;   // first column of this thread
        const uint32_t t_lane = (uint32_t)(quad * 32) << 16;
        const uint32_t tempty0 = mapa_shared(smem_u32(tempty_bar), 0);   // the leader's
        // block scale of K-block kb of B for this warp's 128 columns of tile t (0 outside)
        auto b_scale = [&](const XTile& t, int kb) {
            const int cb = (t.col + col_base) >> 7;
            return kb < t.nkb && cb * 128 < p.cols ? __ldg(p.sb + t.e * p.sb_e + cb * p.sb_c + kb * p.sb_kb) : 0.0f;
        };
        uint32_t acc_it = 0, g_done = 0;
        bool ok = true;
        float sb_cur = 0.0f, sb_nxt = 0.0f;      // lane l: the scale of K-block l of 32
        if ((int)cid < num_items) {
            ok = announced(0);
            if (!WGRAD && ok) sb_nxt = b_scale(told(0), lane);
        }
        uint32_t nt = 0;
        for (int item = (int)cid; ok && item < num_items; item += (int)ncl, ++nt) {
            const bool more = item + (int)ncl < num_items;
            if (more) ok = announced(nt + 1);
            if (!ok) break;
            const int nkb = told(nt).nkb;
            float2 acc[COLS / 2];
            #pragma unroll
            for (int c = 0; c < COLS / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);

            for (int kb = 0; kb < nkb; ++kb, ++acc_it) {
                if (!WGRAD && (kb & 31) == 0) {
                    sb_cur = sb_nxt;
                    if (kb + 32 < nkb) sb_nxt = b_scale(told(nt), kb + 32 + lane);
                    else if (more) sb_nxt = b_scale(told(nt + 1), lane);
                }
                const uint32_t gi = WGRAD ? acc_it : g_done;
                const uint32_t ss = gi % NS;
                const uint32_t ts = acc_it % kBufs;
                const int q = kb % S::SG;
                const bool g_first = q == 0;
                const bool g_last = kb + 1 == nkb || q == S::SG - 1;
                bool got = true;
                if (g_first) got = mbar_wait(smem_u32(&sfull_bar[ss]), (gi / NS) & 1, p.timeout_ns, abort_flag);
                got = got && mbar_wait(smem_u32(&tfull_bar[ts]), (acc_it / kBufs) & 1, p.timeout_ns, abort_flag);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                tc_fence_after();
                const float* slot = ring + ss * S::SLOT;
                if constexpr (WGRAD) {
                    // 16x256b fragments: rows g8 + 8h (h = 0..3) of the warp's 32 and columns
                    // 8j + 2tq + {0,1}; parts of 16 rows x 32 columns, the next part's TMEM
                    // load in flight while this one is promoted
                    const int g8 = lane >> 2, tq = lane & 3;
                    float fr[4];
                    const uint32_t fra = smem_u32(slot) + 4u * (uint32_t)(quad * 32 + g8);
                    #pragma unroll
                    for (int h = 0; h < 4; ++h)
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(fr[h]) : "r"(fra + 32u * h));
                    const uint32_t sba = smem_u32(slot) + 4u * (uint32_t)(S::SLOT_A + col_base + 2 * tq);
                    const uint32_t tb0 = tmem_base + t_lane + ts * kPN + col_base;
                    const uint32_t tb1 = tb0 + (16u << 16);
                    constexpr int NP = 2 * (COLS / 32);
                    uint32_t ra[16], rb[16];
                    float2 sc[4];
                    tmem_ld_16x256b_x4(tb0, ra);
                    tmem_ld_wait(ra);
                    #pragma unroll
                    for (int pp = 0; pp < NP; ++pp) {
                        const int jq = pp >> 1, hh = pp & 1;
                        uint32_t (&cur)[16] = (pp & 1) ? rb : ra;
                        uint32_t (&nxt)[16] = (pp & 1) ? ra : rb;
                        if (pp + 1 < NP) {
                            tmem_ld_16x256b_x4((((pp + 1) & 1) ? tb1 : tb0) + ((pp + 1) >> 1) * 32, nxt);
                        } else {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * ts);
                        }
                        if (hh == 0) {
                            #pragma unroll
                            for (int jj = 0; jj < 4; ++jj)
                                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(sc[jj].x), "=f"(sc[jj].y) : "r"(sba + 32u * (jq * 4 + jj)));
                        }
                        #pragma unroll
                        for (int jj = 0; jj < 4; ++jj) {
                            #pragma unroll
                            for (int h2 = 0; h2 < 2; ++h2) {
                                const int h = 2 * hh + h2;
                                const int o = 4 * jj + 2 * h2;
                                const float2 s2 = __fmul2_rn(make_float2(fr[h], fr[h]), sc[jj]);
                                acc[h * (COLS / 8) + jq * 4 + jj] = __ffma2_rn(make_float2(__uint_as_float(cur[o]), __uint_as_float(cur[o + 1])),
                                                                               s2, acc[h * (COLS / 8) + jq * 4 + jj]);
                            }
                        }
                        if (pp + 1 < NP) tmem_ld_wait(nxt);
                    }
                } else {
                    // 32x32b loads: one row and COLS columns per thread, in two loads (as four of 32 columns
                    // 3.5% slower, and 1% with each in flight during the promotion of the one before)
                    const uint32_t tb = tmem_base + t_lane + ts * kPN + col_base;
                    const float f = slot[q * 128 + quad * 32 + lane] * __shfl_sync(0xffffffffu, sb_cur, kb & 31);
                    const float2 f2 = make_float2(f, f);
                    #pragma unroll
                    for (int g = 0; g < COLS / 64; ++g) {
                        uint32_t r[64];
                        tmem_ld_32x32b_x64(tb + g * 64, r);
                        tmem_ld_wait(r);
                        if (g == COLS / 64 - 1) {
                            // the whole partial is in registers: hand the buffer back to the leader
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * ts);
                        }
                        #pragma unroll
                        for (int j = 0; j < 64; j += 2)
                            acc[g * 32 + j / 2] = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), f2, acc[g * 32 + j / 2]);
                    }
                }
                if (g_last) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sempty_bar[ss]));
                    ++g_done;
                }
            }
            if (!ok) break;

            // ---- the warp's 32 rows x COLS columns go out as BF16 boxes of 32 rows x 64 columns
            // (128-byte swizzle: the 16-byte chunk c of row r sits at chunk c ^ (r & 7)), written by
            // TMA, which clips columns outside C; rows behind the segment (or the expert's result)
            // are not stored.
            const XTile t = told(nt);
            taken(nt);
            const int y0 = t.row + quad * 32;
            const int yc = (WGRAD ? t.e * p.rows : 0) + y0;
            if (lane == 0) bulk_wait_read<0>();      // the previous tile's stores have read the boxes
            __syncwarp();
            #pragma unroll
            for (int b = 0; b < COLS / 64; ++b) {
                const uint32_t buf = smem_u32(stage_c + (ew * (COLS / 64) + b) * 4096);
                if constexpr (WGRAD) {
                    // rows g + 8h, columns 8j + 2tq + {0,1}: an 8 x 8 matrix of the fragment a chunk
                    const int r8 = lane & 7, m4 = lane >> 3;
                    #pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        #pragma unroll
                        for (int c = 0; c < 8; c += 4) {
                            uint32_t v[4];
                            #pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 a = acc[h * (COLS / 8) + b * 8 + c + i];
                                v[i] = pack_bf16x2(a.x, a.y);
                            }
                            st_matrix_x4(buf + (r8 + 8 * h) * 128 + (((c + m4) ^ r8) << 4), v);
                        }
                    }
                } else {
                    #pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int cc = b * 64 + c * 8;    // first of these 8 columns
                        uint4 v;
                        v.x = pack_bf16x2(acc[cc / 2 + 0].x, acc[cc / 2 + 0].y);
                        v.y = pack_bf16x2(acc[cc / 2 + 1].x, acc[cc / 2 + 1].y);
                        v.z = pack_bf16x2(acc[cc / 2 + 2].x, acc[cc / 2 + 2].y);
                        v.w = pack_bf16x2(acc[cc / 2 + 3].x, acc[cc / 2 + 3].y);
                        st_shared_v4(buf + lane * 128 + ((c ^ (lane & 7)) << 4), v);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                #pragma unroll
                for (int b = 0; b < COLS / 64; ++b) {
                    const int x = t.col + col_base + b * 64;
                    if (y0 < t.row_end && x < p.cols)
                        tma_store_2d(&tmC, smem_u32(stage_c + (ew * (COLS / 64) + b) * 4096), x, yc);
                }
                bulk_commit();
            }
        }
        if (lane == 0) bulk_wait_all();   // tile stores complete before exit
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync_all();   // the pair's MMAs and remote arrivals are done in both CTAs
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

template <bool WGRAD>
cudaError_t launch_t(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tsa, const CUtensorMap& tsb,
                     const CUtensorMap& tc, const ExpertGemmParams& p, int clusters, cudaStream_t st) {
    auto kern = k_gemm_experts<WGRAD>;
    const size_t most = XSmem<WGRAD>::bytes((int)kMaxExperts);
    if (most > 227 * 1024) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(2 * clusters), dim3(x_threads(XSmem<WGRAD>::EPI)), XSmem<WGRAD>::bytes(p.E), st, ta, tb, tsa,
                            tsb, tc, p);
}

}  // namespace

// Launch contract (checked by the caller): A's and B's maps have 128 x 128-byte boxes; tsa is A's
// row-scale map with boxes of 128 x min(4, K-blocks) (WGrad: 128 x 1), tsb (WGrad) B's with boxes of
// 256 x 1; tc the BF16 output map (boxes of 64 columns x 32 rows).
cudaError_t launch_gemm_experts(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tsa, const CUtensorMap& tsb,
                                const CUtensorMap& tc, const ExpertGemmParams& p, bool wgrad, int clusters, cudaStream_t st) {
    return wgrad ? launch_t<true>(ta, tb, tsa, tsb, tc, p, clusters, st)
                 : launch_t<false>(ta, tb, tsa, tsb, tc, p, clusters, st);
}

// Reads and clears this translation unit's device status word.  The caller has synchronized the
// stream.
fp8rl_status read_and_clear_experts_status() {
    unsigned int v = 0;
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof v) != cudaSuccess) return FP8RL_ERR_CUDA;
    if (v != 0 && cudaMemcpyToSymbol(g_device_status, &zero, sizeof zero) != cudaSuccess) return FP8RL_ERR_CUDA;
    return static_cast<fp8rl_status>(v);
}

}  // namespace fp8rl
