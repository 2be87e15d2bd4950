// sweep.cuh -- the many-token sweep of the log-probabilities: H W^T on CTA
// pairs, every 256 x 256 tile reduced on chip to its rows' statistics.
//
// The tensor core adds each K = 16 step to its fp32 accumulator with
// truncation, which over thousands of products biases a large logit by many
// ulp (lse 4e-6 off relative at D = 2560, where one fp32 rounding is 6e-8).
// So an accumulator runs over at most 512 products: the two TMEM buffers
// alternate between K segments of one tile, and the epilogue adds each
// finished segment, rounded to nearest, to sums it keeps in registers.
// Relative error of the alternatives' log-probabilities and time of the sweep
// at 4096 x 2560 x 151936, by products per run: 256: 1.5e-7, 3.18 ms; 512:
// 3.0e-7, 2.90 ms; 1024: 5.7e-7, 2.76 ms; all 2560: 1.7e-6, 2.67 ms (whole
// calls).  At logits of 20 and D = 4800, runs of 1024 are twice as far off as
// an fp32 product, runs of 512 as far.  A switch of accumulators costs the
// tensor pipe about 440 cycles, whether or not the epilogue reads anything.
// Eight epilogue warps (two per TMEM lane quadrant, 128 columns each) hold a
// whole tile that way, 128 sums per thread; the registers come from the
// warpgroup that loads and issues (setmaxnreg).
//
// The pipeline is that of umma_gemm.cuh: same tiles, ring, walk and bounded
// waits.
#pragma once
#include "logprob.cuh"

namespace fldce {

constexpr int kSweepThreads = 384;          // warpgroup 0: load, MMA; 1 and 2: epilogue
constexpr int kSegIters = 8;                // K steps of 64 per accumulator run
constexpr int kSliceCols = 128;             // columns per slice (per epilogue thread)

template <int KC>
struct SweepParams {
    float c;                     // |s| log2(e)
    int neg;                     // s < 0: a = -(x W^T + b)
    int64_t V;
    int rows;
    const __nv_bfloat16* bias;   // [V] or null
    LpParts parts;
};

template <class Cfg, int KC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kSweepThreads, 1)
k_logprob_sweep(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const GemmGeom geom, const __grid_constant__ SweepParams<KC> p, int32_t* err) {
    static_assert(Cfg::NSUB == 1 && !Cfg::A_MN && !Cfg::B_MN, "row-major H and W, 256-column tiles");
    constexpr int S = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * Cfg::STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();          // 0 = pair leader
    const uint32_t pair = cluster_id_x();
    const uint32_t npairs = cluster_count_x();
    const uint32_t sbase = smem_u32(smem);
    auto full_bar = [&](int s) { return smem_u32(bars + s); };
    auto empty_bar = [&](int s) { return smem_u32(bars + S + s); };
    auto tfull_bar = [&](int b) { return smem_u32(bars + 2 * S + b); };
    auto tempty_bar = [&](int b) { return smem_u32(bars + 2 * S + 2 + b); };
    const uint32_t drain_bar = smem_u32(bars + 2 * S + 4);   // abort path only

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 16);      // 8 epilogue warps x 2 CTAs
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                            // the peer's barriers exist before use
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int units = geom.num_tiles;
    const int segs = (geom.k_iters + kSegIters - 1) / kSegIters;

    auto fail = [&]() {
        *abort_flag = 1;
        if (lane == 0) atomicOr(err, FLDCE_DEV_ERR_TIMEOUT);
    };

    uint32_t loads_issued = 0;                 // producer: stages loaded so far
    if (warp < 4) {
        // 4 x 32 x 40 + 8 x 32 x 232 = 384 x 168, the launch's registers
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            // -------------------------------------------- TMA producer (both CTAs)
            const uint64_t pol = l2_policy_evict_normal();
            const uint32_t lead_full0 = mapa_shared(full_bar(0), 0);
            uint32_t& it = loads_issued;
            bool ok = true;
            for (int u = pair; ok && u < units && !*abort_flag; u += npairs) {
                int mt, nt, split, k0, k1;
                walk_unit(geom, geom.k_iters, u, mt, nt, split, k0, k1);
                const int arow = mt * Cfg::PAIR_M + (int)rank * Cfg::BM;
                const int brow = nt * Cfg::BN + (int)rank * 128;
                for (int k = 0; k < geom.k_iters; ++k, ++it) {
                    const int s = it % S;
                    if (!mbar_wait_bounded(empty_bar(s), ((it / S) & 1u) ^ 1u, kWaitLimitNs)) {
                        fail();
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        const uint32_t sa = sbase + s * Cfg::STAGE_BYTES;
                        const uint32_t fb = lead_full0 + 8u * (uint32_t)s;
                        if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2 * Cfg::STAGE_BYTES);
                        tma_load_2d_pair(sa, &tmA, fb, k * Cfg::BK, arow, pol);
                        tma_load_2d_pair(sa + Cfg::A_BYTES, &tmB, fb, k * Cfg::BK, brow, pol);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------- MMA issuer (leader)
            uint32_t it = 0, run = 0;          // run: accumulator runs so far
            bool ok = true;
            for (int u = pair; ok && u < units && !*abort_flag; u += npairs) {
                for (int k = 0; k < geom.k_iters; ++run) {
                    const int b = (int)(run & 1u);
                    if (!mbar_wait_bounded(tempty_bar(b), ((run >> 1) & 1u) ^ 1u, kWaitLimitNs)) {
                        fail();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(b * Cfg::BN);
                    const int kend = min(geom.k_iters, k + kSegIters);
                    for (bool first = true; k < kend; ++k, ++it, first = false) {
                        const int s = it % S;
                        if (!mbar_wait_bounded(full_bar(s), (it / S) & 1u, kWaitLimitNs)) {
                            fail();
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (lane == 0) {
                            const uint32_t sa = sbase + s * Cfg::STAGE_BYTES;
                            const uint32_t sb = sa + Cfg::A_BYTES;
#pragma unroll
                            for (int kk = 0; kk < Cfg::BK / 16; ++kk)
                                tc_mma_f16_pair(d_tmem, smem_desc_sw128(sa + kk * 32, 16, 1024),
                                                smem_desc_sw128(sb + kk * 32, 16, 1024), Cfg::IDESC,
                                                (!first || kk > 0) ? 1u : 0u);
                            tc_commit_pair_mc(empty_bar(s), 0x3);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (lane == 0) tc_commit_pair_mc(tfull_bar(b), 0x3);
                    __syncwarp();
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int q = warp & 3;                 // TMEM lane quadrant of this warp
        const int half = (warp - 4) >> 2;       // column half of the tile
        const uint32_t lead_tempty0 = mapa_shared(tempty_bar(0), 0);
        const float c = p.c;
        uint32_t run = 0;
        bool ok = true;
        for (int u = pair; ok && u < units && !*abort_flag; u += npairs) {
            int mt, nt, split, k0, k1;
            walk_unit(geom, geom.k_iters, u, mt, nt, split, k0, k1);
            const int m = mt * Cfg::PAIR_M + (int)rank * Cfg::BM + q * 32 + lane;
            const int64_t n0 = (int64_t)nt * Cfg::BN + half * kSliceCols;
            const bool live = m < p.rows;
            float sum[kSliceCols];
            for (int seg = 0; seg < segs; ++seg, ++run) {
                const int b = (int)(run & 1u);
                if (!mbar_wait_bounded(tfull_bar(b), (run >> 1) & 1u, kWaitLimitNs)) {
                    fail();
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) +
                                    (uint32_t)(b * Cfg::BN + half * kSliceCols);
#pragma unroll
                for (int j = 0; j < kSliceCols / 32; ++j) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(ta + 32u * j, r);
                    tmem_ld_wait_regs(r);
                    if (j == kSliceCols / 32 - 1) {
                        // drained: hand the accumulator back
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(lead_tempty0 + 8u * (uint32_t)b);
                    }
                    if (seg == 0) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[32 * j + i] = __uint_as_float(r[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            add2(sum[32 * j + i], sum[32 * j + i + 1], sum[32 * j + i],
                                 sum[32 * j + i + 1], __uint_as_float(r[i]),
                                 __uint_as_float(r[i + 1]));
                    }
                }
            }
            if (!ok) break;
            const int64_t left = p.V - n0;
            if (left <= 0) continue;            // a slice past the vocabulary
            const int ncols = (int)(left < kSliceCols ? left : kSliceCols);
            RunningStats rs;
            ThreadTop<KC> tt;
            if constexpr (KC > 0) tt.init(live ? row_floor<KC>(p.parts, m) : CUDART_INF_F);
#pragma unroll
            for (int j = 0; j < kSliceCols / 32; ++j) {
                float a[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) a[i] = sum[32 * j + i];
                if (p.bias != nullptr) {
                    float bv[32];
                    load_bias32(p.bias, n0 + 32 * j, p.V, bv);
#pragma unroll
                    for (int i = 0; i < 32; ++i) a[i] += bv[i];
                }
                if (p.neg) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) a[i] = -a[i];
                }
                if (32 * j + 32 > ncols) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * j + i >= ncols) a[i] = -CUDART_INF_F;
                }
                float cm0 = fmaxf(a[0], a[1]), cm1 = fmaxf(a[2], a[3]);
#pragma unroll
                for (int i = 4; i < 32; i += 4) {
                    cm0 = fmax3(cm0, a[i], a[i + 1]);
                    cm1 = fmax3(cm1, a[i + 2], a[i + 3]);
                }
                const float cm = fmaxf(cm0, cm1);
                const float ref = rs.rebase(fmaxf(rs.m, cm), c);
                float l0 = 0.f, l1 = 0.f, w0 = 0.f, w1 = 0.f;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float d0, d1;
                    add2(d0, d1, a[i], a[i + 1], -ref, -ref);
                    mul2(d0, d1, d0, d1, c, c);
                    // a may be -inf (a bias, a weight, past the vocabulary):
                    // 2^d d is 0 then, not 0 * inf (a NaN stays one in 2^d)
                    const float e0 = ex2(d0), e1 = ex2(d1);
                    add2(l0, l1, l0, l1, e0, e1);
                    fma2(w0, w1, e0, e1, fmaxf(d0, -1e4f), fmaxf(d1, -1e4f), w0, w1);
                }
                rs.l += l0 + l1;
                rs.w += w0 + w1;
                if constexpr (KC > 0) {
                    if (cm > tt.v[KC - 1]) {
                        uint32_t mask = 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i) mask |= (a[i] > tt.v[KC - 1] ? 1u : 0u) << i;
                        while (mask != 0) {
                            const int i = __ffs(mask) - 1;
                            mask &= mask - 1;
                            const float x = select32(a, i);
                            if (x > tt.v[KC - 1]) tt.insert(x, (int)n0 + 32 * j + i);
                        }
                    }
                }
            }
            if (live) store_part<KC>(p.parts, (int)(n0 / kSliceCols), m, rs, tt);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // as in umma_gemm.cuh: what was issued completes before TMEM is freed
        // and the CTAs exit (each wait bounded again)
        if (rank == 0 && warp == 1 && lane == 0) {
            tc_commit_pair_mc(drain_bar, 0x1);
            mbar_wait_bounded(drain_bar, 0u, kWaitLimitNs);
        }
        if (rank == 0 && warp == 0 && lane == 0) {
            const uint32_t first = loads_issued > (uint32_t)S ? loads_issued - S : 0u;
            for (uint32_t i = first; i < loads_issued; ++i)
                mbar_wait_bounded(full_bar((int)(i % S)), (i / S) & 1u, kWaitLimitNs);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    }
    cluster_sync();            // every MMA of the pair has completed and been read
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    }
}

}  // namespace fldce
