// logprob_host.cuh -- host side of the token log-probabilities and of the
// 4-bit head weight (fldce_logprob*, fldce_w4_*).  Included by fldce_api.cu,
// whose launch helpers it uses.
//
// Forward, per chunk of tokens: a sweep leaves every vocabulary slice's
// statistics and candidates, k_logprob_merge joins them.  Backward, per chunk:
// k_logprob_coef turns the upstream gradients into row coefficients, one
// sweep recomputes the logits into G, and the training path's dH and dW
// products follow.
#pragma once

namespace {

// Partial statistics of one forward chunk: at most this much workspace.
constexpr size_t kLpBudget = size_t(1) << 30;
constexpr int64_t kW4ChunkTokens = 256;         // tokens of a forward chunk on a 4-bit weight

// TMA loads from a tensor map that spans less than 128 KiB in all run at a
// fraction of their speed (measured, whatever the box, pitch or alignment: a
// sweep over 32000 x 1024 takes 58 us for 63 tokens and 24 us for 64), so
// fewer hidden states than that are copied and padded with zero rows.
constexpr size_t kSmallMap = size_t(128) << 10;
bool pads_rows(int64_t rows, int64_t D) { return (size_t)rows * D * 2 < kSmallMap; }
int64_t padded_rows(int64_t D) { return cdiv((int64_t)kSmallMap, 2 * D); }

// fldce_selftest_device_error: the device error bits that calls start from.
std::atomic<int32_t> g_selftest_dev_err{0};

cudaError_t clear_counters(Counters* cnt, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(cnt, 0, sizeof(Counters), st);
    const int32_t bits = g_selftest_dev_err.load(std::memory_order_relaxed);
    if (e == cudaSuccess && bits != 0) e = cudaMemsetAsync(&cnt->dev_err, bits & 0xff, 1, st);
    return e;
}

// H [rows, D] bf16 as the maps should see it: itself, or its padded copy in buf.
cudaError_t pad_rows(const void** H, int64_t* map_rows, void* buf, int64_t rows, int64_t D,
                     cudaStream_t st) {
    *map_rows = rows;
    if (!pads_rows(rows, D)) return cudaSuccess;
    *map_rows = padded_rows(D);
    const int64_t n = *map_rows * (D / 8);
    k_pad_rows<<<(unsigned)cdiv(n, 256), 256, 0, st>>>(static_cast<const uint4*>(*H),
                                                       rows * (D / 8), static_cast<uint4*>(buf), n);
    *H = buf;
    return cudaGetLastError();
}

struct LpLayout {
    size_t cnt, stats, top, floor, hpad, total;
    int64_t C;                // tokens per chunk
    int64_t n_parts;
    int kc;
    bool few;                 // k_few instead of the tensor-core sweep's 256-row tiles
};

LpLayout lp_layout(const fldce_plan* p, int64_t N, int top_k, bool w4) {
    LpLayout L{};
    L.kc = candidates_for(top_k);
    L.few = w4 || (p->cfg.dtype == FLDCE_BF16 && N <= kFewTokens);
    L.n_parts = L.few ? kFewMaxParts : cdiv(p->cfg.V, p->cfg.dtype == FLDCE_BF16 ? kSliceCols : kSimtTile);
    const size_t per_row = (size_t)L.n_parts * (16 + 8 * (size_t)L.kc);
    int64_t C = std::max<int64_t>(256, (int64_t)(kLpBudget / per_row) / 256 * 256);
    if (w4) C = kW4ChunkTokens;
    L.C = std::max<int64_t>(1, std::min(C, N));
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = round_up(off + bytes, kAlign);
        return o;
    };
    L.cnt = take(sizeof(Counters));
    L.stats = take((size_t)L.n_parts * L.C * 16);
    L.top = take((size_t)L.n_parts * L.C * L.kc * 8);
    L.floor = take((size_t)L.C * 4 * (L.kc + 1));
    L.hpad = take((size_t)padded_rows(p->cfg.D) * p->cfg.D * 2);
    L.total = off;
    return L;
}

// Workspace of the gradient.  G has room for whole 32-row store boxes; dH of
// few tokens or columns, whose product has few tiles, may be split over K
// more often than the loss's, up to 16 ways while the partials stay small.
constexpr int kLpColsumSegs = 16;               // row segments of db's column sums
constexpr int kLpSplits = 16;
constexpr int64_t kLpSplitBytes = int64_t(64) << 20;
int lp_max_splits(int64_t C, int64_t D) {
    const int64_t part = (int64_t)round_up((size_t)C, 256) * D * 4;
    return (int)std::max<int64_t>(kMaxKSplits, std::min<int64_t>(kLpSplits, kLpSplitBytes / part));
}
// Room for that many partials, without the steps of the division: it grows with C.
size_t lp_split_bytes(int64_t C, int64_t D) {
    const int64_t part = (int64_t)round_up((size_t)C, 256) * D * 4;
    return (size_t)std::max(kMaxKSplits * part, std::min(kLpSplits * part, kLpSplitBytes));
}

// G of up to this many tokens is in two bf16 terms, 2 rows each (as many as
// the 32 rows that G always has room for).  One rounding to bf16 is as large
// as the results' own: where one or two elements make up most of a row, dH, dW
// and db of 1 to 16 tokens were up to 2.5 times as far off as once-rounded
// results (20,000 random steps; now 1.002 times).  Over more tokens it
// averages out: at most 1.48 times with 17 to 64, so those keep one term.
// The products' 256-row tiles and their 64-wide K step have the room.
constexpr int kTwoTermTokens = 16;

struct LpBwdLayout : Layout {
    size_t hpad, repeats;
};

LpBwdLayout lp_bwd_layout(const fldce_plan* p, int64_t N) {
    LpBwdLayout L{};
    const int64_t C = std::max<int64_t>(1, std::min<int64_t>(p->chunk, N));
    L.C = C;
    L.nchunks = N > 0 ? cdiv(N, p->chunk) : 0;
    const bool bf16 = p->cfg.dtype == FLDCE_BF16;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = round_up(off + bytes, kAlign);
        return o;
    };
    L.cnt = take(sizeof(Counters));
    L.zy = take(C * 4);
    L.row_lse2 = take(C * 4);
    L.row_gcoef = take(C * 4);
    L.row_y = take(C * 4);
    L.loss_tok = take(C * 4);
    L.part_sz = take(C * 4);
    L.part_am = take(bf16 ? C * 4 : 0);
    L.part_ml = take(bf16 ? (size_t)p->cfg.V * 4 : 0);
    L.G = take(round_up((size_t)C, 32) * p->Vpad * p->elt);
    L.dh_acc = take(bf16 ? lp_split_bytes(C, p->cfg.D) : 0);
    const bool acc = (L.nchunks > 1 || (dw_accumulate(p) && N > 0)) && !dw_out_fp32(p);
    L.dw_acc = take(acc ? (size_t)p->cfg.V * p->cfg.D * 4 : 0);
    L.db_part = take((size_t)kLpColsumSegs * p->cfg.V * 4);
    L.db_acc = take((size_t)p->cfg.V * 4);
    L.hpad = take(bf16 ? (size_t)std::max<int64_t>(padded_rows(p->cfg.D), 2 * kTwoTermTokens) * p->cfg.D * 2
                       : 0);
    L.repeats = take(bf16 ? (size_t)std::min(C, p->cfg.V) * p->cfg.D * 4 : 0);
    L.total = off;
    return L;
}

// Shapes every 4-bit weight has to have.
int check_w4(const void* packed, const void* scales, int group, int64_t V, int64_t D) {
    if (V <= 0 || D <= 0) return FLDCE_ERR_INVALID_ARG;
    if (packed == nullptr || scales == nullptr) return FLDCE_ERR_INVALID_ARG;
    if (D % 32 != 0 || (group != 32 && group != 64 && group != 128)) return FLDCE_ERR_UNSUPPORTED;
    if (V > (int64_t(1) << 31) - 1 || D > (int64_t(1) << 31) - 1) return FLDCE_ERR_UNSUPPORTED;
    if (!aligned16(packed) || !aligned_to(scales, 2)) return FLDCE_ERR_ALIGN;
    return FLDCE_OK;
}

HeadWeight w4_weight(const void* packed, const void* scales, int group, int64_t D) {
    return HeadWeight{packed, static_cast<const __nv_bfloat16*>(scales), group,
                      (int)cdiv(D, group)};
}

// Set a kernel's shared-memory limit once per device (as launch_gemm does).
template <class K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& done) {
    int devid = 0;
    cudaError_t e = cudaGetDevice(&devid);
    if (e != cudaSuccess) return e;
    const uint64_t bit = devid < 64 ? (uint64_t(1) << devid) : 0;
    if (bit == 0 || (done.load(std::memory_order_acquire) & bit) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

// How the vocabulary is cut for k_few: one range of rows per CTA, in full
// tiles and a last one.
struct FewGrid {
    int ctas, cta_rows, tiles, last_rows;
};

FewGrid few_grid(int64_t V, int sms) {
    FewGrid g;
    const int n = std::min(std::max(sms, 1), kFewMaxParts);
    g.cta_rows = (int)round_up((size_t)cdiv(V, n), 8);
    g.ctas = (int)cdiv(V, g.cta_rows);
    g.tiles = (int)cdiv(g.cta_rows, kFewRows);
    g.last_rows = g.cta_rows - (g.tiles - 1) * kFewRows;
    return g;
}

template <bool W4, int LB, int NT, int KC>
cudaError_t launch_few_nt(FewParams& p, const FewGrid& g, const HeadWeight& hw,
                          const __nv_bfloat16* x, int64_t D, cudaStream_t st) {
    using Cfg = FewCfg<W4, LB, NT>;
    p.k_stages = (int)cdiv(D, Cfg::KS);
    const bool maps =
        make_map(&p.xmap, x, D, p.n_tok, D, 64, 8 * NT) &&
        (W4 ? make_map(&p.wmap, hw.W, D / 2, p.V, D / 2, 128, kFewRows, 1) &&
                  make_map(&p.wmap_last, hw.W, D / 2, p.V, D / 2, 128, g.last_rows, 1)
            : make_map(&p.wmap, hw.W, D, p.V, D, 64, kFewRows) &&
                  make_map(&p.wmap_last, hw.W, D, p.V, D, 64, g.last_rows));
    if (!maps) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    auto kern = k_few<W4, LB, NT, KC>;
    if (cudaError_t e = allow_smem(kern, Cfg::SMEM_BYTES, done)) return e;
    kern<<<g.ctas, Cfg::THREADS, Cfg::SMEM_BYTES, st>>>(p);
    return cudaGetLastError();
}

template <bool W4, int LB, int KC>
cudaError_t launch_few_lb(FewParams& p, const FewGrid& g, const HeadWeight& hw,
                          const __nv_bfloat16* x, int64_t D, cudaStream_t st) {
    if (p.n_tok <= 8) return launch_few_nt<W4, LB, 1, KC>(p, g, hw, x, D, st);
    if (p.n_tok <= 16) return launch_few_nt<W4, LB, 2, KC>(p, g, hw, x, D, st);
    if (p.n_tok <= 24) return launch_few_nt<W4, LB, 3, KC>(p, g, hw, x, D, st);
    return launch_few_nt<W4, LB, 4, KC>(p, g, hw, x, D, st);
}

// One pass over the weight for up to kFewTokens tokens.
template <bool W4, int KC>
cudaError_t launch_few(FewParams& p, const HeadWeight& hw, const __nv_bfloat16* x, int64_t D,
                       int sms, cudaStream_t st) {
    const FewGrid g = few_grid(p.V, sms);
    p.cta_rows = g.cta_rows;
    p.tiles = g.tiles;
    p.last_rows = g.last_rows;
    p.hw = hw;
    p.broken = g_selftest_dev_err.load(std::memory_order_relaxed);
    if constexpr (W4) {
        if (hw.group == 32) return launch_few_lb<true, 0, KC>(p, g, hw, x, D, st);
        if (hw.group == 64) return launch_few_lb<true, 1, KC>(p, g, hw, x, D, st);
        return launch_few_lb<true, 2, KC>(p, g, hw, x, D, st);
    } else {
        return launch_few_lb<false, 0, KC>(p, g, hw, x, D, st);
    }
}

template <int KC>
cudaError_t launch_sweep(const CUtensorMap& h, const CUtensorMap& w, int rows, int64_t V, int64_t D,
                         const SweepParams<KC>& sp, int32_t* err, int sms, cudaStream_t st) {
    using Cfg = CfgKK;
    GemmGeom g{};
    g.tiles_m = (int)cdiv(rows, Cfg::PAIR_M);
    g.tiles_n = (int)cdiv(V, Cfg::BN);
    g.k_iters = (int)cdiv(D, Cfg::BK);
    g.k_splits = 1;
    g.num_tiles = g.tiles_m * g.tiles_n;
    g.n_fastest = 0;
    g.group = walk_group(g.tiles_m, (size_t)Cfg::PAIR_M * D * 2, kL2BudgetSweep);
    static std::atomic<uint64_t> done{0};
    auto kern = k_logprob_sweep<Cfg, KC>;
    constexpr size_t smem = 1024 + Cfg::STAGES * Cfg::STAGE_BYTES + Cfg::BAR_BYTES;
    if (cudaError_t e = allow_smem(kern, smem, done)) return e;
    const int pairs = std::min(g.num_tiles, std::max(1, sms / 2));
    kern<<<2 * pairs, kSweepThreads, smem, st>>>(h, w, g, sp, err);
    return cudaGetLastError();
}

template <int KC>
int lp_forward(fldce_plan* h, const fldce_logprob_call& call, const LpLayout& L,
               const DeviceInfo& dev) {
    const fldce_config& cfg = h->cfg;
    const int64_t D = cfg.D, V = cfg.V, N = call.N;
    const bool bf16 = cfg.dtype == FLDCE_BF16, w4 = call.w4 != nullptr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(call.stream);
    uint8_t* ws = static_cast<uint8_t*>(call.workspace);
    Counters* cnt = reinterpret_cast<Counters*>(ws + L.cnt);
    LpParts parts{reinterpret_cast<float4*>(ws + L.stats), reinterpret_cast<float2*>(ws + L.top),
                  L.few ? nullptr : reinterpret_cast<uint32_t*>(ws + L.floor), (int)L.C};
    const float c = fabsf(cfg.logit_scale) * 1.4426950408889634f;
    const int neg = cfg.logit_scale < 0.f ? 1 : 0;
    HeadWeight hw{call.W, nullptr, 0, 0};
    if (w4) hw = w4_weight(call.w4, call.w4_scales, call.w4_group, D);
    CUtensorMap mW;
    if (bf16 && !w4 && !make_map(&mW, call.W, D, V, D, 64, 128)) return FLDCE_ERR_CUDA;
    for (int64_t r0 = 0; r0 < N; r0 += L.C) {
        const int rows = (int)std::min<int64_t>(L.C, N - r0);
        const uint8_t* Hc = static_cast<const uint8_t*>(call.H) + (size_t)r0 * D * h->elt;
        if (KC > 0 && !L.few)
            FLDCE_CUDA(cudaMemsetAsync(parts.floor, 0, (size_t)L.C * 4 * (KC + 1), st));
        prof_mark(h, PK_GAP, st);
        if (L.few) {
            const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(Hc);
            FewParams fp{};
            fp.V = V;
            fp.bias = static_cast<const __nv_bfloat16*>(call.bias);
            fp.c = c;
            fp.neg = neg;
            fp.parts = parts;
            fp.err = &cnt->dev_err;
            for (int t0 = 0; t0 < rows; t0 += kFewTokens) {
                fp.n_tok = std::min(kFewTokens, rows - t0);
                fp.row0 = t0;
                if (w4)
                    FLDCE_CUDA((launch_few<true, KC>(fp, hw, x + (int64_t)t0 * D, D, dev.sms, st)));
                else
                    FLDCE_CUDA((launch_few<false, KC>(fp, hw, x + (int64_t)t0 * D, D, dev.sms, st)));
            }
        } else if (bf16) {
            CUtensorMap mH;
            const void* Hm = Hc;
            int64_t map_rows;
            FLDCE_CUDA(pad_rows(&Hm, &map_rows, ws + L.hpad, rows, D, st));
            if (!make_map(&mH, Hm, D, map_rows, D, 64, 128)) return FLDCE_ERR_CUDA;
            const SweepParams<KC> sp{
                c, neg, V, rows, static_cast<const __nv_bfloat16*>(call.bias), parts};
            FLDCE_CUDA(launch_sweep<KC>(mH, mW, rows, V, D, sp, &cnt->dev_err, dev.sms, st));
        } else {
            SimtLogprob<KC> e{fabsf(cfg.logit_scale), c, neg, V, rows,
                              static_cast<const float*>(call.bias), parts};
            FLDCE_CUDA(launch_simt<true>(reinterpret_cast<const float*>(Hc), D, 1,
                                   static_cast<const float*>(call.W), D, 1, rows, V, (int)D, e,
                                   st));
        }
        prof_mark(h, PK_LSE, st);
        LpMergeParams mp{};
        mp.parts = parts;
        mp.n_parts = L.few ? few_grid(V, dev.sms).ctas : (int)L.n_parts;
        mp.D = D;
        mp.V = V;
        mp.ignore_index = cfg.ignore_index;
        mp.s = cfg.logit_scale;
        mp.c = c;
        mp.H = Hc;
        mp.hw = hw;
        mp.bias = call.bias;
        mp.token = call.token != nullptr ? call.token + r0 : nullptr;
        mp.k = call.top_k;
        mp.logprob = call.logprob != nullptr ? call.logprob + r0 : nullptr;
        mp.entropy = call.entropy != nullptr ? call.entropy + r0 : nullptr;
        mp.lse = call.lse != nullptr ? call.lse + r0 : nullptr;
        mp.lse_lo = call.lse != nullptr && (cfg.flags & FLDCE_FLAG_LSE_PAIR) != 0
                        ? call.lse + N + r0 : nullptr;
        mp.top_ids = KC > 0 ? call.top_ids + r0 * call.top_k : nullptr;
        mp.top_logprobs = KC > 0 ? call.top_logprobs + r0 * call.top_k : nullptr;
        mp.n_err = call.err_count;
        // (k_few's statistics are NaN where it failed)
        mp.dev_err = bf16 && !L.few ? &cnt->dev_err : nullptr;
        // a few rows: the latency of one is the kernel's
        if (!bf16)
            k_logprob_merge<KC, float, 128><<<rows, 128, 0, st>>>(mp);
        else if (rows <= kFewTokens) {
            // behind k_few: launched early, its set-up hidden in that kernel's end
            cudaLaunchAttribute early{};
            early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            early.val.programmaticStreamSerializationAllowed = 1;
            cudaLaunchConfig_t lc{};
            lc.gridDim = dim3((unsigned)rows);
            lc.blockDim = dim3(512);
            lc.stream = st;
            lc.attrs = &early;
            lc.numAttrs = 1;
            FLDCE_CUDA(cudaLaunchKernelEx(&lc, k_logprob_merge<KC, __nv_bfloat16, 512>, mp));
        } else
            k_logprob_merge<KC, __nv_bfloat16, 128><<<rows, 128, 0, st>>>(mp);
        FLDCE_CUDA(cudaGetLastError());
        prof_mark(h, PK_MERGE, st);
    }
    // the device error bits of the sweeps
    if (call.err_count != nullptr)
        FLDCE_CUDA(cudaMemcpyAsync(call.err_count + 1, &cnt->dev_err, 4, cudaMemcpyDeviceToDevice,
                                   st));
    return FLDCE_OK;
}

// What the log-probability entry points accept of a plan.
int check_lp_plan(const fldce_plan* h) {
    if (h->sharded || (h->cfg.flags & (FLDCE_FLAG_SKIP_IGNORED | FLDCE_FLAG_FUSED_DH)) != 0)
        return FLDCE_ERR_UNSUPPORTED;
    return FLDCE_OK;
}

}  // namespace

extern "C" {

int fldce_logprob_workspace_size(fldce_handle h, int64_t N, int32_t top_k, size_t* bytes) {
    if (h == nullptr || bytes == nullptr || N < 0 || N > h->cfg.max_N) return FLDCE_ERR_INVALID_ARG;
    if (top_k < 0 || top_k > FLDCE_MAX_TOP_K || top_k > h->cfg.V) return FLDCE_ERR_INVALID_ARG;
    if (int e = check_lp_plan(h)) return e;
    *bytes = std::max(lp_layout(h, N, top_k, false).total, lp_layout(h, N, top_k, true).total);
    return FLDCE_OK;
}

int fldce_logprob(fldce_handle h, const fldce_logprob_call* cp) {
    if (h == nullptr || cp == nullptr) return FLDCE_ERR_INVALID_ARG;
    const fldce_logprob_call& c = *cp;
    if (int e = check_lp_plan(h)) return e;
    const bool w4 = c.w4 != nullptr;
    if (c.N < 0 || c.N > h->cfg.max_N || c.top_k < 0 || c.top_k > FLDCE_MAX_TOP_K ||
        c.top_k > h->cfg.V)
        return FLDCE_ERR_INVALID_ARG;
    if ((c.W != nullptr) == w4) return FLDCE_ERR_INVALID_ARG;
    if (c.N > 0 && c.H == nullptr) return FLDCE_ERR_INVALID_ARG;
    if (c.logprob != nullptr && c.token == nullptr) return FLDCE_ERR_INVALID_ARG;
    if (c.N > 0 && c.top_k > 0 && (c.top_ids == nullptr || c.top_logprobs == nullptr))
        return FLDCE_ERR_INVALID_ARG;
    if (w4) {
        if (h->cfg.dtype != FLDCE_BF16) return FLDCE_ERR_UNSUPPORTED;
        if (int e = check_w4(c.w4, c.w4_scales, c.w4_group, h->cfg.V, h->cfg.D)) return e;
    }
    if (c.workspace == nullptr || !aligned_to(c.workspace, kAlign)) return FLDCE_ERR_WORKSPACE;
    if (!aligned16(c.H) || !aligned16(c.W) || !aligned16(c.bias)) return FLDCE_ERR_ALIGN;
    if (!aligned_to(c.token, 8) || !aligned_to(c.logprob, 4) || !aligned_to(c.entropy, 4) ||
        !aligned_to(c.lse, 4) || !aligned_to(c.top_ids, 4) || !aligned_to(c.top_logprobs, 4) ||
        !aligned_to(c.err_count, 4))
        return FLDCE_ERR_ALIGN;
    const LpLayout L = lp_layout(h, c.N, c.top_k, w4);
    if (c.workspace_bytes < L.total) return FLDCE_ERR_WORKSPACE;
    DeviceInfo dev;
    if (int s = check_device(&dev)) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(c.stream);
    Counters* cnt = reinterpret_cast<Counters*>(static_cast<uint8_t*>(c.workspace) + L.cnt);
    if (c.err_count != nullptr) FLDCE_CUDA(cudaMemsetAsync(c.err_count, 0, 8, st));
    // (k_few's error bits are only reported: without err_count nobody reads them)
    if (c.err_count != nullptr || (h->cfg.dtype == FLDCE_BF16 && !L.few))
        FLDCE_CUDA(clear_counters(cnt, st));
    if (c.N == 0) return FLDCE_OK;
    switch (L.kc) {
        case 0: return lp_forward<0>(h, c, L, dev);
        case candidates_for(1): return lp_forward<candidates_for(1)>(h, c, L, dev);
        case candidates_for(5): return lp_forward<candidates_for(5)>(h, c, L, dev);
        case candidates_for(12): return lp_forward<candidates_for(12)>(h, c, L, dev);
        default: return lp_forward<candidates_for(FLDCE_MAX_TOP_K)>(h, c, L, dev);
    }
}

int fldce_logprob_bwd_workspace_size(fldce_handle h, int64_t N, size_t* bytes) {
    if (h == nullptr || bytes == nullptr || N < 0 || N > h->cfg.max_N) return FLDCE_ERR_INVALID_ARG;
    if (int e = check_lp_plan(h)) return e;
    *bytes = lp_bwd_layout(h, N).total;
    return FLDCE_OK;
}

int fldce_logprob_bwd(fldce_handle h, const fldce_logprob_grad_call* cp) {
    if (h == nullptr || cp == nullptr) return FLDCE_ERR_INVALID_ARG;
    const fldce_logprob_grad_call& c = *cp;
    if (int e = check_lp_plan(h)) return e;
    const fldce_config& cfg = h->cfg;
    const int64_t N = c.N, D = cfg.D, V = cfg.V;
    if (N < 0 || N > cfg.max_N) return FLDCE_ERR_INVALID_ARG;
    if (c.dH == nullptr && c.dW == nullptr && c.db == nullptr && N > 0) return FLDCE_ERR_INVALID_ARG;
    if (N > 0 && (c.H == nullptr || c.W == nullptr || c.lse == nullptr)) return FLDCE_ERR_INVALID_ARG;
    if (N > 0 && c.dlogprob != nullptr && c.token == nullptr) return FLDCE_ERR_INVALID_ARG;
    if (N > 0 && c.dentropy != nullptr && c.entropy == nullptr) return FLDCE_ERR_INVALID_ARG;
    if (c.db != nullptr && c.bias == nullptr) return FLDCE_ERR_INVALID_ARG;
    if (c.workspace == nullptr || !aligned_to(c.workspace, kAlign)) return FLDCE_ERR_WORKSPACE;
    if (!aligned16(c.H) || !aligned16(c.W) || !aligned16(c.bias) || !aligned16(c.dH) ||
        !aligned16(c.dW) || !aligned16(c.db))
        return FLDCE_ERR_ALIGN;
    if (!aligned_to(c.token, 8) || !aligned_to(c.lse, 4) || !aligned_to(c.entropy, 4) ||
        !aligned_to(c.dlogprob, 4) || !aligned_to(c.dentropy, 4) || !aligned_to(c.err_count, 4))
        return FLDCE_ERR_ALIGN;
    const LpBwdLayout L = lp_bwd_layout(h, N);
    if (c.workspace_bytes < L.total) return FLDCE_ERR_WORKSPACE;
    DeviceInfo dev;
    if (int s = check_device(&dev)) return s;

    cudaStream_t st = reinterpret_cast<cudaStream_t>(c.stream);
    uint8_t* ws = static_cast<uint8_t*>(c.workspace);
    Counters* cnt = reinterpret_cast<Counters*>(ws + L.cnt);
    const bool bf16 = cfg.dtype == FLDCE_BF16, accum = dw_accumulate(h);
    const size_t dw_elt = dw_out_fp32(h) ? 4 : h->elt;
    const float c2 = cfg.logit_scale * 1.4426950408889634f;
    if (c.err_count != nullptr) {
        FLDCE_CUDA(cudaMemsetAsync(c.err_count, 0, 8, st));
        FLDCE_CUDA(clear_counters(cnt, st));
    }
    if (N == 0) {
        if (!accum && c.dW != nullptr)
            FLDCE_CUDA(cudaMemsetAsync(c.dW, 0, (size_t)V * D * dw_elt, st));
        if (!accum && c.db != nullptr) FLDCE_CUDA(cudaMemsetAsync(c.db, 0, (size_t)V * dw_elt, st));
        return FLDCE_OK;
    }
    LpCoef k{reinterpret_cast<float*>(ws + L.row_lse2), reinterpret_cast<float*>(ws + L.row_gcoef),
             reinterpret_cast<float*>(ws + L.zy), reinterpret_cast<float*>(ws + L.loss_tok),
             reinterpret_cast<int32_t*>(ws + L.row_y), reinterpret_cast<float*>(ws + L.part_sz),
             nullptr, reinterpret_cast<int32_t*>(ws + L.part_am)};
    float* repeats = reinterpret_cast<float*>(ws + L.repeats);
    const float* lse_lo = (cfg.flags & FLDCE_FLAG_LSE_PAIR) != 0 ? c.lse + N : nullptr;
    float* db_part = reinterpret_cast<float*>(ws + L.db_part);
    float* db_acc = reinterpret_cast<float*>(ws + L.db_acc);
    CUtensorMap mW_k, mW_mn;
    if (bf16 && (!make_map(&mW_k, c.W, D, V, D, 64, 128) || !make_map(&mW_mn, c.W, D, V, D, 64, 64)))
        return FLDCE_ERR_CUDA;
    prof_mark(h, PK_GAP, st);
    for (int64_t ci = 0; ci < L.nchunks; ++ci) {
        const int64_t r0 = ci * h->chunk;
        const int rows = (int)std::min<int64_t>(h->chunk, N - r0);
        const uint8_t* Hc = static_cast<const uint8_t*>(c.H) + (size_t)r0 * D * h->elt;
        const bool few = bf16 && rows <= kFewTokens, two = bf16 && rows <= kTwoTermTokens;
        const int g_rows = two ? 2 * rows : rows;       // (H's rows twice to match)
        const bool pads = bf16 && (two || pads_rows(rows, D));
        const int64_t map_rows =
            pads_rows(g_rows, D) ? std::max<int64_t>(padded_rows(D), g_rows) : g_rows;
        k.first = bf16 && !two && c.dW != nullptr ? reinterpret_cast<int32_t*>(ws + L.part_ml)
                                                  : nullptr;
        const int64_t n_pad = pads ? map_rows * (D / 8) : 0;
        uint4* hp = reinterpret_cast<uint4*>(ws + L.hpad);
        const int64_t n_thr = std::max({k.first != nullptr ? std::max<int64_t>(V, 32 * (int64_t)rows)
                                                           : (int64_t)rows, n_pad});
        k_logprob_coef<<<(unsigned)cdiv(n_thr, 256), 256, 0, st>>>(
            c.token != nullptr ? c.token + r0 : nullptr, c.lse + r0,
            c.entropy != nullptr ? c.entropy + r0 : nullptr,
            c.dlogprob != nullptr ? c.dlogprob + r0 : nullptr,
            c.dentropy != nullptr ? c.dentropy + r0 : nullptr, rows, V, cfg.ignore_index,
            cfg.logit_scale, k, c.err_count, reinterpret_cast<const uint4*>(Hc), rows * (D / 8), hp,
            n_pad, two ? 2 : 1, !bf16, lse_lo != nullptr ? lse_lo + r0 : nullptr,
            ci == 0 ? &cnt->dev_err : nullptr, g_selftest_dev_err.load(std::memory_order_relaxed));
        FLDCE_CUDA(cudaGetLastError());
        prof_mark(h, PK_MERGE, st);
        void* G = ws + L.G;
        if (bf16) {
            CUtensorMap mH_k, mH_mn, mG_k, mG_mn;
            LogprobGEpi::Params gp;
            const void* Hm = pads ? static_cast<const void*>(hp) : Hc;
            // (whole boxes of rows: rows past the tokens get zeros)
            if (!make_store_map(&gp.gmap, G, V, round_up((size_t)rows, 32), h->Vpad, 2) ||
                !make_map(&mH_k, Hm, D, map_rows, D, 64, 128) ||
                !make_map(&mH_mn, Hm, D, map_rows, D, 64, 64) ||
                !make_map(&mG_k, G, V, g_rows, h->Vpad, 64, 128) ||
                !make_map(&mG_mn, G, V, g_rows, h->Vpad, 64, 64))
                return FLDCE_ERR_CUDA;
            gp.c = c2;
            gp.V = V;
            gp.rows = rows;
            gp.k = k;
            gp.bias = static_cast<const __nv_bfloat16*>(c.bias);
            if (few) {
                FewParams fp{};
                fp.V = V;
                fp.bias = gp.bias;
                fp.n_tok = rows;
                fp.out = G;
                fp.ldo = h->Vpad;
                fp.two_terms = two ? 1 : 0;
                fp.c2 = c2;
                fp.k = k;
                fp.err = &cnt->dev_err;
                FLDCE_CUDA((launch_few<false, -2>(fp, HeadWeight{c.W, nullptr, 0, 0},
                                                  reinterpret_cast<const __nv_bfloat16*>(Hc), D,
                                                  dev.sms, st)));
            } else {
                const Walk walk{0, 1, walk_group(cdiv(rows, CfgKK::PAIR_M),
                                                 (size_t)CfgKK::PAIR_M * D * 2, kL2BudgetSweep)};
                FLDCE_CUDA((launch_gemm<CfgKK, LogprobGEpi>(mH_k, mW_k, rows, V, D, walk, gp,
                                                            &cnt->dev_err, dev.sms, st)));
            }
            prof_mark(h, PK_G, st);
            GradGemm gg{h,  &L,   ws, cnt,       &dev,
                        st, g_rows, r0, DynRows(), lp_max_splits(L.C, D)};
            if (two) {
                gg.fold_tokens = rows;
            } else {
                gg.dh_rest = RowRest{k.y, nullptr, k.res, static_cast<const __nv_bfloat16*>(c.W), (int)V};
                gg.dw_rest = RowRest{k.first, k.next, k.res, reinterpret_cast<const __nv_bfloat16*>(Hc),
                                     rows, repeats, V <= L.C};
            }
            if (c.dH != nullptr)
                if (int e = gg.dh(mG_k, mW_mn, c.dH)) return e;
            if (c.dW != nullptr) {
                if (!two && c.token != nullptr) {
                    const unsigned blocks = (unsigned)std::min<int64_t>(rows, 4 * (int64_t)dev.sms);
                    k_logprob_repeats<<<dim3(blocks, (unsigned)cdiv(D, 1024)), 128, 0, st>>>(
                        k, rows, reinterpret_cast<const __nv_bfloat16*>(Hc), D, V <= L.C, repeats);
                    FLDCE_CUDA(cudaGetLastError());
                }
                if (int e = gg.dw(mG_mn, mH_mn, c.dW, ci)) return e;
            }
        } else {
            const float* Hf = reinterpret_cast<const float*>(Hc);
            const float* Wf = static_cast<const float*>(c.W);
            float* Gf = static_cast<float*>(G);
            SimtLogprobG ge{cfg.logit_scale, V, h->Vpad, rows, k, Gf, static_cast<const float*>(c.bias)};
            FLDCE_CUDA(launch_simt<true>(Hf, D, 1, Wf, D, 1, rows, V, (int)D, ge, st));
            prof_mark(h, PK_G, st);
            if (c.dH != nullptr) {
                SimtStore hs{rows, D, D, static_cast<float*>(c.dH) + r0 * D, nullptr, 0};
                FLDCE_CUDA(launch_simt<true>(Gf, h->Vpad, 1, Wf, 1, D, rows, D, (int)V, hs, st));
                prof_mark(h, PK_DH, st);
            }
            if (c.dW != nullptr) {
                float* dw = static_cast<float*>(c.dW);
                const int mode = accum ? 2 : (L.nchunks == 1 ? 0 : (ci == 0 ? 1 : 2));
                SimtStore wsd{(int)V, D, D, dw, dw, mode};
                FLDCE_CUDA(launch_simt<true>(Gf, 1, h->Vpad, Hf, 1, D, (int)V, D, rows, wsd, st));
                prof_mark(h, PK_DW, st);
            }
        }
        if (c.db != nullptr) {
            int nseg = (int)std::min<int64_t>(kLpColsumSegs, cdiv(g_rows, 32));
            if (bf16) {
                const dim3 grid((unsigned)cdiv(V, 512), (unsigned)nseg);
                k_logprob_colsum<<<grid, 128, 0, st>>>(static_cast<const __nv_bfloat16*>(G),
                                                       h->Vpad, g_rows, V, (int)cdiv(g_rows, nseg),
                                                       db_part);
                FLDCE_CUDA(cudaGetLastError());
            } else {
                FLDCE_CUDA(launch_colsum_partial(G, false, h->Vpad, rows, V, db_part, st, 32,
                                                 &nseg));
            }
            const bool last = ci + 1 == L.nchunks;
            k_logprob_db<<<(unsigned)cdiv(V, 256), 256, 0, st>>>(
                db_part, nseg, V, k.y, k.res, bf16 && !two ? rows : 0, db_acc, ci > 0 ? 1 : 0,
                last ? c.db : nullptr, dw_out_fp32(h) ? 0 : 1, accum ? 1 : 0);
            FLDCE_CUDA(cudaGetLastError());
            prof_mark(h, PK_DB, st);
        }
    }
    if (bf16) {
        const size_t dh_elt = (cfg.flags & FLDCE_FLAG_DH_FP32) != 0 ? 4 : 2;
        k_logprob_void<<<dev.sms, 512, 0, st>>>(
            &cnt->dev_err, static_cast<uint4*>(c.dH),
            c.dH != nullptr ? (int64_t)((size_t)N * D * dh_elt / 16) : 0,
            static_cast<uint4*>(c.dW), c.dW != nullptr ? (int64_t)((size_t)V * D * dw_elt / 16) : 0,
            static_cast<uint16_t*>(c.db), c.db != nullptr ? (int64_t)(V * dw_elt / 2) : 0);
        FLDCE_CUDA(cudaGetLastError());
    }
    if (c.err_count != nullptr)
        FLDCE_CUDA(cudaMemcpyAsync(c.err_count + 1, &cnt->dev_err, 4, cudaMemcpyDeviceToDevice,
                                   st));
    return FLDCE_OK;
}

int fldce_selftest_device_error(int32_t bits) {
    if (bits < 0 || bits > 0xff) return FLDCE_ERR_INVALID_ARG;
    g_selftest_dev_err.store(bits, std::memory_order_relaxed);
    return FLDCE_OK;
}

int fldce_w4_quantize(const void* W, int32_t dtype, int64_t V, int64_t D, int32_t group,
                      void* packed, void* scales, void* stream) {
    if (W == nullptr) return FLDCE_ERR_INVALID_ARG;
    if (dtype != FLDCE_BF16 && dtype != FLDCE_FP32) return FLDCE_ERR_UNSUPPORTED;
    if (int e = check_w4(packed, scales, group, V, D)) return e;
    if (!aligned16(W)) return FLDCE_ERR_ALIGN;
    DeviceInfo dev;
    if (int s = check_device(&dev)) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int blocks = (int)std::min<int64_t>(cdiv(V * cdiv(D, group), 8), 16 * (int64_t)dev.sms);
    uint8_t* q = static_cast<uint8_t*>(packed);
    __nv_bfloat16* sc = static_cast<__nv_bfloat16*>(scales);
    if (dtype == FLDCE_BF16)
        k_w4_quantize<<<blocks, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(W), V, D, group, q,
                                              sc);
    else
        k_w4_quantize<<<blocks, 256, 0, st>>>(static_cast<const float*>(W), V, D, group, q, sc);
    return cudaGetLastError() == cudaSuccess ? FLDCE_OK : FLDCE_ERR_CUDA;
}

int fldce_w4_linear(const void* x, int64_t N, const void* packed, const void* scales, int32_t group,
                    const void* bias, int64_t V, int64_t D, void* out, int32_t out_dtype,
                    int32_t* err_count, void* stream) {
    if (N < 0 || N > (int64_t(1) << 31) - 1) return FLDCE_ERR_INVALID_ARG;
    if (out_dtype != FLDCE_BF16 && out_dtype != FLDCE_FP32) return FLDCE_ERR_UNSUPPORTED;
    if (int e = check_w4(packed, scales, group, V, D)) return e;
    if (N > 0 && (x == nullptr || out == nullptr)) return FLDCE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned_to(bias, 2) || !aligned_to(err_count, 4) ||
        !aligned_to(out, out_dtype == FLDCE_BF16 ? 2 : 4))
        return FLDCE_ERR_ALIGN;
    DeviceInfo dev;
    if (int s = check_device(&dev)) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (err_count != nullptr) FLDCE_CUDA(cudaMemsetAsync(err_count, 0, 8, st));
    const HeadWeight hw = w4_weight(packed, scales, group, D);
    const size_t row_bytes = (size_t)V * (out_dtype == FLDCE_BF16 ? 2 : 4);
    FewParams fp{};
    fp.V = V;
    fp.bias = static_cast<const __nv_bfloat16*>(bias);
    fp.out_bf16 = out_dtype == FLDCE_BF16 ? 1 : 0;
    fp.err = err_count != nullptr ? err_count + 1 : nullptr;
    for (int64_t t0 = 0; t0 < N; t0 += kFewTokens) {
        fp.n_tok = (int)std::min<int64_t>(kFewTokens, N - t0);
        fp.out = static_cast<uint8_t*>(out) + t0 * row_bytes;
        FLDCE_CUDA((launch_few<true, -1>(fp, hw, static_cast<const __nv_bfloat16*>(x) + t0 * D, D,
                                         dev.sms, st)));
    }
    return FLDCE_OK;
}

}  // extern "C"
