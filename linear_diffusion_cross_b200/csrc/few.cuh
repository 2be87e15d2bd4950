// few.cuh -- the head's product for few tokens (up to 32 at a time), with a
// 16-bit or a 4-bit weight: its logits, or their statistics without them.
//
// The weight is streamed once: the vocabulary is cut into one contiguous range
// of rows per SM, a multiple of 8 rows, so nearly every SM reads the same
// bytes and there is no last round (the last range gets what is left, 232 of
// 1032 rows at V = 151936; rounding up to 8 leaves SMs without one where V is
// small, 73 of 148 at V = 1200).  With 16-bit weights and few tokens the
// weight's bytes bound it (4 tokens of 2560 x 151936: 125 us, 119 at the
// measured copy rate); with 4 bits, or more tokens, the instructions do.
// A producer thread keeps a ring of TMA boxes in flight (up to 198 KB
// per SM, several times bandwidth x latency) across tile boundaries; 8 or
// 16 consumer warps turn them into logits with m16n8k16 matrix instructions:
// vocabulary rows are M and tokens are N, so one token costs an 8-column
// product, where the 256-row tiles of the many-token sweep would spend 256.
// A warp takes 32 rows (two M tiles share the token operand) and, up to 16
// tokens, one half of each stage's K; the halves meet in shared memory at the
// end of a tile.
//
// 4-bit weights go from shared memory to registers as 32-bit words of eight
// nibbles.  (w >> 4 i) & 0x000f000f holds elements i and i + 4; or-ing them
// into the mantissa of 128 (with the sign bit flipped) gives 136 + q in
// bf16, and a subtraction of 136 is exact: the products are of integers.
// The token operand is paired to match (elements i and i + 4) by byte
// permutes.  A group's sum is scaled in fp32 when the group ends; with groups
// of 32, 64 or 128 every 32-element block lies in one group.
//
// Sums are kept short: the matrix instruction truncates its fp32 accumulator
// at every step, so a run of at most 128 products (or a group) is added to
// the row's sum by a rounded fp32 addition.
#pragma once
#include "w4.cuh"

namespace fldce {

// Tokens per pass, and the most that this kernel takes from the 256-row tiles
// of a 16-bit weight.  Log-probabilities with one alternative, here against
// there, in us:  tokens of   2560 x 151936   2048 x 32000   3920 x 159722
//                       8      137 / 195        37 / 65
//                      24      160 / 198        41 / 61
//                      32      174 / 188        44 / 58        244 / 334
// and the gradient's G:  8     142 / 172        31 / 45
//                      32      170 / 170        36 / 45        249 / 332
constexpr int kFewTokens = 32;
constexpr int kFewRows = 256;           // rows of a tile at most
constexpr int kFewMaxParts = 160;       // CTAs at most

template <bool W4, int LB, int NT>
struct FewCfg {
    static constexpr int KS = W4 ? 256 : 64;                  // elements of K per stage
    // Consumer warps: eight 32-row groups, by two K halves while the token
    // operand and the sums leave room in the registers.
    static constexpr int HALVES = NT <= 2 ? 2 : 1;
    static constexpr int CONSUMERS = 8 * HALVES;
    static constexpr int THREADS = 32 * (CONSUMERS + 1);
    static constexpr int XBOXES = KS / 64;                    // 64-element boxes of x
    static constexpr uint32_t W_BYTES = kFewRows * 128;       // a box row is 128 bytes
    static constexpr uint32_t XBOX_BYTES = 8 * NT * 128;
    static constexpr int NG = W4 ? 8 >> LB : 0;               // scales per row and stage
    static constexpr uint32_t SCALE_BYTES = W4 ? kFewRows * NG * 2 : 0;
    static constexpr uint32_t SCALE_OFF = W_BYTES + XBOXES * XBOX_BYTES;
    static constexpr uint32_t STAGE_BYTES = SCALE_OFF + SCALE_BYTES;
    // the logits of a tile: [token][row]; the pitch spreads a fragment's
    // store over all banks
    static constexpr int PITCH = kFewRows + (W4 ? 8 : 4);
    static constexpr uint32_t LG_BYTES = 8 * NT * PITCH * 4;
    static constexpr int STAGES =
        (int)((232448u - 1024u - 256u - LG_BYTES) / STAGE_BYTES) < 6
            ? (int)((232448u - 1024u - 256u - LG_BYTES) / STAGE_BYTES) : 6;
    static constexpr uint32_t SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + LG_BYTES + 256;
    static constexpr int TPW = (8 * NT + CONSUMERS - 1) / CONSUMERS;   // tokens per warp
    static_assert(STAGES >= 3 && STAGE_BYTES % 1024 == 0 && SMEM_BYTES <= 232448, "shared memory");
};

struct FewParams {
    CUtensorMap wmap;          // [V, D] boxes of kFewRows x 128 bytes, 128B swizzle
    CUtensorMap wmap_last;     // the same in boxes of last_rows
    CUtensorMap xmap;          // [n_tok, D] bf16 boxes of 8 NT x 64, 128B swizzle
    int64_t V;
    // Vocabulary rows per CTA (a multiple of 8), in tiles of kFewRows and a
    // last one of last_rows: full tiles occupy every warp.
    int cta_rows;
    int tiles;
    int last_rows;
    int k_stages;              // ceil(D / KS)
    int n_tok;
    HeadWeight hw;             // scales of a 4-bit weight
    const __nv_bfloat16* bias; // [V] or null
    // statistics
    float c;                   // |s| log2(e)
    int neg;                   // s < 0
    LpParts parts;             // rows row0 .. row0 + n_tok - 1
    int row0;
    // logits, or their gradient
    void* out;                 // [n_tok][V] (gradient: bf16, rows ldo apart)
    int out_bf16;
    int64_t ldo;
    int two_terms;             // the gradient in two terms, 2 n_tok rows
    float c2;                  // s log2(e)
    LpCoef k;                  // the gradient's row coefficients
    int32_t* err;              // device error bits, or null
    int broken;                // act as if a wait had run out (the self-test's)
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                            int32_t x, int32_t y, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (a & mask) ^ flip in one logic instruction.
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t flip) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(a), "r"(mask), "r"(flip));
    return d;
}

// Pairs (i, i + 4), i = 0..3, of a word of eight nibbles, as bf16.
__device__ __forceinline__ void nibble_pairs(uint32_t w, uint32_t (&r)[4]) {
    const __nv_bfloat162 off = __halves2bfloat162(__ushort_as_bfloat16(0x4308),
                                                  __ushort_as_bfloat16(0x4308));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = and_xor(w >> (4 * i), 0x000f000fu, 0x43084308u);   // 136 + q
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), off);
        r[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

// Copy N bytes (4, 8 or 16) global -> shared asynchronously.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N)
                 : "memory");
}
// Arrive on `bar` when this thread's copies so far have landed (the barrier's
// count includes the arrival).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, unsigned short v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// N 16-bit values at addr, two to a word.
template <int N>
__device__ __forceinline__ void ld_shared_u16s(uint32_t addr, uint32_t (&w)[(N + 1) / 2]) {
    if constexpr (N == 1) {
        unsigned short h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
        w[0] = h;
    } else if constexpr (N == 2) {
        w[0] = ld_shared_u32(addr);
    } else if constexpr (N == 4) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr)
                     : "memory");
    } else {
        const uint4 v = ld_shared_v4(addr);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// KC >= 0: statistics and KC candidates per (CTA, token).  -1: logits.
// -2: the logits' gradient (as LogprobGEpi).
// LB: log2 of a 4-bit weight's group in 32-element blocks.
template <bool W4, int LB, int NT, int KC>
__global__ void __launch_bounds__(FewCfg<W4, LB, NT>::THREADS, 1)
k_few(const __grid_constant__ FewParams p) {
    using Cfg = FewCfg<W4, LB, NT>;
    constexpr int S = Cfg::STAGES;
    constexpr int HALVES = Cfg::HALVES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* lg = reinterpret_cast<float*>(smem + S * Cfg::STAGE_BYTES);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * Cfg::STAGE_BYTES + Cfg::LG_BYTES);
    const uint32_t sbase = smem_u32(smem);
    auto full_bar = [&](int s) { return smem_u32(bars + s); };
    auto empty_bar = [&](int s) { return smem_u32(bars + S + s); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), W4 ? 33 : 1);             // the boxes; 32 lanes' scales
            mbar_init(empty_bar(s), Cfg::CONSUMERS);
        }
        fence_mbar_init();
        tma_prefetch_desc(&p.wmap);
        tma_prefetch_desc(&p.wmap_last);
        tma_prefetch_desc(&p.xmap);
    }
    __syncthreads();
    // the merge may be made ready to start (it waits for this grid to end)
    if (KC >= 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t r_begin = (int64_t)blockIdx.x * p.cta_rows;
    const int64_t r_end = min(p.V, r_begin + p.cta_rows);

    if (warp == Cfg::CONSUMERS) {
        // ------------------------------------------------ producer
        const uint64_t pol_w = l2_policy_evict_first();         // read once
        const uint64_t pol_x = l2_policy_evict_normal();
        // scales of a row and stage as one asynchronous copy where they are
        // aligned for it (D a multiple of 256), else element by element
        const bool whole = W4 && p.hw.groups % (W4 ? Cfg::NG : 1) == 0 &&
                           (reinterpret_cast<uintptr_t>(p.hw.scales) % (2 * Cfg::NG + !W4)) == 0;
        int s = 0, it = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int t = 0; ok && t < p.tiles; ++t) {
            const int64_t row0 = r_begin + (int64_t)t * kFewRows;
            const bool last = t + 1 == p.tiles;
            const CUtensorMap* wmap = last ? &p.wmap_last : &p.wmap;
            const int tile_rows = last ? p.last_rows : kFewRows;
            const uint32_t bytes = (uint32_t)tile_rows * 128u + Cfg::XBOXES * Cfg::XBOX_BYTES;
            const unsigned short* src[W4 ? 8 : 1];           // scales of rows lane + 32 i
            if constexpr (W4) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    src[i] = reinterpret_cast<const unsigned short*>(p.hw.scales) +
                             min(row0 + lane + 32 * i, p.V - 1) * p.hw.groups;
            }
            for (int k = 0; k < p.k_stages; ++k, ++it) {
                if (!mbar_wait_bounded(empty_bar(s), ph, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                const uint32_t sw = sbase + s * Cfg::STAGE_BYTES;
                if (lane == 0) {
                    mbar_arrive_expect_tx(full_bar(s), bytes);
                    // a box row is 128 bytes: 64 bf16, or 256 nibbles (128 one-byte columns)
                    tma_load_2d(sw, wmap, full_bar(s), k * (W4 ? 128 : 64), (int)row0, pol_w);
#pragma unroll
                    for (int b = 0; b < Cfg::XBOXES; ++b)
                        tma_load_2d(sw + Cfg::W_BYTES + b * Cfg::XBOX_BYTES, &p.xmap, full_bar(s),
                                    k * Cfg::KS + 64 * b, 0, pol_x);
                }
                if constexpr (W4) {
                    __syncwarp();
                    const uint32_t dst = sw + Cfg::SCALE_OFF + (uint32_t)lane * 2 * Cfg::NG;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (32 * i >= tile_rows) break;
                        const uint32_t d = dst + (uint32_t)(64 * i * Cfg::NG);
                        if (whole) {
                            cp_async<2 * Cfg::NG>(d, src[i]);
                            src[i] += Cfg::NG;
                        } else {
#pragma unroll
                            for (int j = 0; j < Cfg::NG; ++j)
                                st_shared_u16(d + 2 * j, __ldg(src[i] + min(k * Cfg::NG + j,
                                                                           p.hw.groups - 1)));
                        }
                    }
                    if (whole) cp_async_arrive(full_bar(s));
                    else mbar_arrive(full_bar(s));
                }
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        if (!ok) {
            if (lane == 0 && p.err != nullptr) atomicOr(p.err, FLDCE_DEV_ERR_TIMEOUT);
            // loads in flight land before the CTA may exit (bounded again)
            for (int i = it > S ? it - S : 0; i < it; ++i)
                mbar_wait_bounded(full_bar(i % S), (i / S) & 1u, kWaitLimitNs);
        }
        return;
    }

    // ---------------------------------------------------- consumers
    const int rg = warp / HALVES, half = warp % HALVES;     // 32-row group, K half
    const int g = lane >> 2, t4 = lane & 3;
    bool ok = true;
    // A tile's logits of a token are read by `wpt` warps (a power of two, one
    // when there are more tokens than warps), each a slice of its 32-row runs.
    int wpt = 1;
    while (2 * wpt * p.n_tok <= Cfg::CONSUMERS) wpt *= 2;
    const int tok0 = warp / wpt, slice = warp % wpt;
    RunningStats rs[Cfg::TPW];
    WarpTop<(KC > 0 ? KC : 1)> wt[Cfg::TPW];

    constexpr int NB = 8 / HALVES;                          // 32-element blocks per stage
    constexpr int NS = W4 ? NB >> LB : 1;                   // scales per row and stage half

    // shared-memory offsets within a stage, the 128-byte swizzle included
    uint32_t w_off[W4 ? 4 : 1], x_off[2];
    const uint32_t h4 = (uint32_t)half * 4u;                // first 16-byte chunk of the half
    // token of product column g: 0 4 1 5 2 6 3 7 (4-bit), so that the eight
    // lanes of a 16-byte load phase hit eight different chunks
    const uint32_t tok_g = W4 ? (uint32_t)(((g & 1) << 2) + (g >> 1)) : (uint32_t)(lane & 7);
    if constexpr (W4) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
            w_off[b] = (uint32_t)(rg * 32 + g) * 128u + (((h4 + b) ^ g) << 4) + 4u * t4;
        x_off[0] = Cfg::W_BYTES + (uint32_t)(half * 2) * Cfg::XBOX_BYTES + tok_g * 128u +
                   (((uint32_t)t4 ^ tok_g) << 4);
        x_off[1] = Cfg::W_BYTES + (uint32_t)(half * 2) * Cfg::XBOX_BYTES + tok_g * 128u +
                   (((uint32_t)(4 + t4) ^ tok_g) << 4);
    } else {
        const uint32_t row = (uint32_t)(rg * 32 + (lane & 15));
        w_off[0] = row * 128u;
        x_off[0] = Cfg::W_BYTES + tok_g * 128u;
        x_off[1] = 0;
    }

    int s = 0;
    uint32_t ph = 0;
    for (int t = 0; t < p.tiles; ++t) {
        const int tile_rows = t + 1 == p.tiles ? p.last_rows : kFewRows;
        const bool active = rg * 32 < tile_rows;
        float acc[2][NT][4], part[2][NT][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][n][e] = part[m][n][e] = 0.f;
        for (int k = 0; k < p.k_stages; ++k) {
                if (ok && !mbar_wait_bounded(full_bar(s), ph, kWaitLimitNs)) {
                    ok = false;
                    if (lane == 0 && p.err != nullptr) atomicOr(p.err, FLDCE_DEV_ERR_TIMEOUT);
                }
                if (!ok) continue;
            if (active) {
                const uint32_t st = sbase + s * Cfg::STAGE_BYTES;
                if constexpr (W4) {
                    // scales of this thread's rows (8 i + g of the group), two to a word
                    uint32_t sc[4][(NS + 1) / 2];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ld_shared_u16s<NS>(st + Cfg::SCALE_OFF +
                                               (uint32_t)((rg * 32 + 8 * i + g) * Cfg::NG +
                                                          half * NS) * 2, sc[i]);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        // one half: blocks 4..7 sit in the other four chunks
                        const uint32_t wa = st + (b < 4 ? w_off[b & 3] : w_off[b & 3] ^ 64u);
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)          // rows 8 i + g of the group
                            w[i] = ld_shared_u32(wa + 1024u * i);
                        uint32_t a[2][2][4];                 // [M tile][k16 step]
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            uint32_t lo[4], hi[4];           // rows g and g + 8
                            nibble_pairs(w[2 * m], lo);
                            nibble_pairs(w[2 * m + 1], hi);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                a[m][q][0] = lo[2 * q];
                                a[m][q][1] = hi[2 * q];
                                a[m][q][2] = lo[2 * q + 1];
                                a[m][q][3] = hi[2 * q + 1];
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 x = ld_shared_v4(st + x_off[b & 1] +
                                                         (b >> 1) * Cfg::XBOX_BYTES + n * 1024u);
                            const uint32_t p0 = __byte_perm(x.x, x.z, 0x5410);
                            const uint32_t p1 = __byte_perm(x.x, x.z, 0x7632);
                            const uint32_t p2 = __byte_perm(x.y, x.w, 0x5410);
                            const uint32_t p3 = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                mma_bf16(part[m][n], a[m][0], p0, p1);
                                mma_bf16(part[m][n], a[m][1], p2, p3);
                            }
                        }
                        if (((b + 1) & ((1 << LB) - 1)) == 0) {
                            // the group ends: scale its integer products
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const int j = b >> LB;
                                const uint32_t w0 = sc[2 * m][j / 2], w1 = sc[2 * m + 1][j / 2];
                                const float s0 = __uint_as_float((j & 1) ? w0 & 0xffff0000u : w0 << 16);
                                const float s1 = __uint_as_float((j & 1) ? w1 & 0xffff0000u : w1 << 16);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        acc[m][n][e] = fmaf(part[m][n][e], e < 2 ? s0 : s1,
                                                            acc[m][n][e]);
                                        part[m][n][e] = 0.f;
                                    }
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int q2 = 0; q2 < 2 / HALVES; ++q2) {        // 32 elements of K
                        const uint32_t c0 = h4 + 4u * q2;            // first 16-byte chunk
                        uint32_t b[NT][4];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            ldmatrix_x4(st + x_off[0] + n * 1024u +
                                            (((c0 + (lane >> 3)) ^ (lane & 7)) << 4), b[n]);
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                uint32_t a[4];
                                ldmatrix_x4(st + w_off[0] + 2048u * m +
                                                (((c0 + 2u * q + (lane >> 4)) ^ (lane & 7)) << 4),
                                            a);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma_bf16(part[m][n], a, b[n][2 * q], b[n][2 * q + 1]);
                            }
                    }
                    if ((k & (2 * HALVES - 1)) == 2 * HALVES - 1 || k + 1 == p.k_stages) {
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    acc[m][n][e] += part[m][n][e];
                                    part[m][n][e] = 0.f;
                                }
                    }
                }
            }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_bar(s));
                if (++s == S) { s = 0; ph ^= 1u; }
        }
        if (!ok || p.broken) {
            // a wait ran out: these rows are NaN, not the sum of what came
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][n][e] = CUDART_NAN_F;
        }
        // the tile's logits, the K halves added: lg[token][row]
        auto cell = [&](int m, int n, int e) -> float* {
            const int row = rg * 32 + 16 * m + g + (e >= 2 ? 8 : 0);
            const int col = 2 * t4 + (e & 1);               // column of the product
            const int tok = 8 * n + (W4 ? ((col & 1) << 2) + (col >> 1) : col);
            return lg + tok * Cfg::PITCH + row;
        };
        if (active && half == HALVES - 1) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) *cell(m, n, e) = acc[m][n][e];
        }
        // this lane's rows of the tile, and their bias (asked for before the
        // barrier): i = 32 (slice + wpt j) + lane
        const int64_t v0 = r_begin + (int64_t)t * kFewRows;
        const int rows = (int)max((int64_t)0, min((int64_t)tile_rows, r_end - v0));
        const int js = 8 / min(wpt, 8);                     // 32-row runs of a warp
        float bias[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = 32 * (slice + wpt * j) + lane;
            bias[j] = p.bias != nullptr && i < rows ? __bfloat162float(__ldg(p.bias + v0 + i)) : 0.f;
        }
        consumers_sync<32 * Cfg::CONSUMERS>();
        if (HALVES == 2 && active && half == 0) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) *cell(m, n, e) += acc[m][n][e];
        }
        if (HALVES == 2) consumers_sync<32 * Cfg::CONSUMERS>();
#pragma unroll
        for (int q = 0; q < Cfg::TPW; ++q) {
            const int tok = tok0 + q * Cfg::CONSUMERS;
            if (tok >= p.n_tok) continue;
            const float* src = lg + tok * Cfg::PITCH;
            float a[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = 32 * (slice + wpt * j) + lane;
                a[j] = i < rows ? src[i] + bias[j] : kNegInf;
            }
            if constexpr (KC == -2) {
                // bf16; in two terms, what that took off goes to row n_tok + tok
                const float L2 = p.k.lse2[tok], kap = p.k.kap[tok], ee = p.k.ee[tok];
                const float ta = p.k.ta[tok];
                const int64_t y = p.k.y[tok];
                const bool dead = kap == 0.f && ee == 0.f && ta == 0.f;
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (int64_t)tok * p.ldo + v0;
                __nv_bfloat16* o2 = o + (int64_t)p.n_tok * p.ldo;
                const bool two = p.two_terms != 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 32 * (slice + wpt * j) + lane;
                    if (i >= rows) continue;
                    float gr = lp_grad(fmaf(a[j], p.c2, -L2), kap, ee);
                    if (dead) gr = 0.f;
                    else if (v0 + i == y) {
                        gr += ta;
                        if (!two) {
                            p.k.res[tok] = bf16_rest(gr);
                            if (p.k.first != nullptr) atomicMin(p.k.first + y, tok);
                        }
                    }
                    o[i] = __float2bfloat16_rn(gr);
                    if (two) o2[i] = __float2bfloat16_rn(bf16_rest(gr));
                }
            } else if constexpr (KC < 0) {
                const int64_t o = (int64_t)tok * p.V + v0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 32 * (slice + wpt * j) + lane;
                    if (i >= rows) continue;
                    if (p.out_bf16)
                        static_cast<__nv_bfloat16*>(p.out)[o + i] = __float2bfloat16_rn(a[j]);
                    else
                        static_cast<float*>(p.out)[o + i] = a[j];
                }
            } else {
                if (p.neg) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        a[j] = 32 * (slice + wpt * j) + lane < rows ? -a[j] : kNegInf;
                }
                float mx = rs[q].m;
#pragma unroll
                for (int j = 0; j < 8; ++j) mx = fmaxf(mx, a[j]);
                const float ref = rs[q].rebase(mx, p.c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j >= js) break;
                    rs[q].add(a[j], ref, p.c);
                    if constexpr (KC > 0)
                        wt[q].offer(a[j], (int)(v0 + 32 * (slice + wpt * j) + lane), lane);
                }
            }
        }
        consumers_sync<32 * Cfg::CONSUMERS>();              // lg is free again
    }
    if constexpr (KC >= 0) {
        // a warp's lanes, then a token's warps (through lg), become one part
        float* sm_stats = lg;                               // [warp][3]
        uint64_t* sm_key = reinterpret_cast<uint64_t*>(lg + 4 * Cfg::CONSUMERS);  // [warp][32]
#pragma unroll
        for (int j = 0; j < Cfg::TPW; ++j) {
            const int tok = tok0 + j * Cfg::CONSUMERS;
            const bool mine = tok < p.n_tok;
            float mx = rs[j].m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            rs[j].rebase(mx, p.c);
            float l = rs[j].l, w = rs[j].w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, o);
                w += __shfl_xor_sync(0xffffffffu, w, o);
            }
            if (wpt > 1) {
                if (j > 0) break;                           // a warp has one token then
                if (lane == 0) {
                    sm_stats[3 * warp] = mx;
                    sm_stats[3 * warp + 1] = l;
                    sm_stats[3 * warp + 2] = w;
                }
                if (KC > 0) sm_key[32 * warp + lane] = lane < KC ? wt[j].key : 0;
                consumers_sync<32 * Cfg::CONSUMERS>();
                if (!mine || slice != 0) continue;
                float ml = kNegInf, ll = 0.f, wl = 0.f;     // lane i < wpt: the i-th warp's
                if (lane < wpt) {
                    ml = sm_stats[3 * (warp + lane)];
                    ll = sm_stats[3 * (warp + lane) + 1];
                    wl = sm_stats[3 * (warp + lane) + 2];
                }
                mx = ml;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                RunningStats r;
                r.m = ml;
                r.l = ll;
                r.w = wl;
                r.rebase(mx, p.c);
                l = r.l;
                w = r.w;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    l += __shfl_xor_sync(0xffffffffu, l, o);
                    w += __shfl_xor_sync(0xffffffffu, w, o);
                }
                if constexpr (KC > 0)
                    for (int i = 1; i < wpt; ++i)
                        wt[j].offer_key(sm_key[32 * (warp + i) + lane], lane);
            }
            if (!mine) continue;
            const size_t part = blockIdx.x;
            const int row = p.row0 + tok;
            int n = 0;
            if constexpr (KC > 0) {
                const bool has = lane < KC && wt[j].key != 0;
                n = __popc(__ballot_sync(0xffffffffu, has));
                if (has)
                    p.parts.top[(part * KC + lane) * p.parts.ld + row] =
                        make_float2(rank_value(wt[j].key), __int_as_float(rank_id(wt[j].key)));
            }
            if (lane == 0)
                p.parts.stats[part * p.parts.ld + row] = make_float4(mx, l, w, __int_as_float(n));
        }
    }
}

}  // namespace fldce
