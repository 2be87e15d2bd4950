// logprob.cuh -- device code of the token log-probabilities: log p of given
// tokens, entropy, the best alternatives, and the gradient of both.
//
// With z = s (x W^T + b) and p = softmax(z):
//   lse = log sum_v e^(z_v),  logprob = z_y - lse,  entropy = lse - sum_v p_v z_v.
// Any slice of the vocabulary is summarised by
//   m = max a,  l = sum 2^d,  w = sum 2^d d,   a = sign(s) (x W^T + b),  d = c (a - m),
//   c = |s| log2(e),
// and slices merge exactly: with f = 2^(c (m - M)), l -> f l and
// w -> f (w + c (m - M) l).  At the end lse = c M ln 2 + ln l and
// entropy = ln l - ln 2 w / l, a difference of small numbers (lse - sum p z
// would cancel).  The maximum is taken before the scale, so that logits of
// the type's lowest value keep their differences instead of overflowing.
//
// The alternatives' order is decided in 64 bits: every slice keeps its KC best
// columns by the fp32 accumulator, the merge keeps the KC best of all slices
// (KC exceeds the k asked for by 3 or more), recomputes their dot products in
// fp64 and sorts by (value, lowest id).  So ids do not depend on the summation
// order of the matrix instructions, the tile that computed them, or the
// number of tokens in the call, unless more than KC - k columns past the k-th
// come within the fp32 error of it: which KC of them are kept is fp32's choice.
#pragma once
#include "kernels.cuh"

namespace fldce {

constexpr float kNegInf = -__builtin_huge_valf();

// Candidates kept per slice for k alternatives.
constexpr int candidates_for(int k) {
    return k == 0 ? 0 : (k == 1 ? 4 : (k <= 5 ? 8 : (k <= 12 ? 16 : 24)));
}

// Order-preserving map of floats to unsigned integers (0 is below every
// float; -0 counts as +0).
__device__ __forceinline__ uint32_t float_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The running (m, l, w) of one row over a slice, fed in groups of values.
struct RunningStats {
    float m = kNegInf, l = 0.f, w = 0.f;

    // Move the reference to nm >= m; returns the finite reference to subtract.
    // (While m is -inf, l and w are 0, or NaN, and stay so.)
    __device__ __forceinline__ float rebase(float nm, float c) {
        const float ref = nm == -CUDART_INF_F ? 0.f : nm;
        if (m != -CUDART_INF_F) {
            const float d = fmaxf((m - nm) * c, -1e4f);   // finite: 2^d d is 0, not 0 * inf
            const float f = ex2(d);
            w = f * fmaf(d, l, w);
            l *= f;
        }
        m = nm;
        return ref;
    }
    __device__ __forceinline__ void add(float a, float ref, float c) {
        float d = (a - ref) * c;
        d = d < -1e4f ? -1e4f : d;          // -inf: 2^d d must be 0 (NaN stays NaN)
        const float e = ex2(d);
        l += e;
        w = fmaf(e, d, w);
    }
};

// KC best (value, column) pairs of one thread, sorted; equal values keep the
// lower column when columns are offered in increasing order.
template <int KC>
struct ThreadTop {
    float v[KC];
    int id[KC];

    // Only values above `floor` are kept.
    __device__ __forceinline__ void init(float floor) {
#pragma unroll
        for (int i = 0; i < KC; ++i) { v[i] = floor; id[i] = -1; }
    }
    __device__ __forceinline__ void insert(float x, int col) {
#pragma unroll
        for (int i = KC - 1; i > 0; --i) {
            const bool shift = x > v[i - 1];
            const bool here = x > v[i];
            id[i] = shift ? id[i - 1] : (here ? col : id[i]);
            v[i] = shift ? v[i - 1] : (here ? x : v[i]);
        }
        if (x > v[0]) { v[0] = x; id[0] = col; }
    }
    __device__ __forceinline__ int count() const {
        int n = 0;
#pragma unroll
        for (int i = 0; i < KC; ++i) n += id[i] >= 0 ? 1 : 0;
        return n;
    }
};

template <>
struct ThreadTop<0> {};

// a[i] for a run-time i without leaving the registers: five levels of selects.
__device__ __forceinline__ float select32(const float (&a)[32], int i) {
    float t[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) t[j] = (i & 16) ? a[j + 16] : a[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = (i & 8) ? t[j + 8] : t[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = (i & 4) ? t[j + 4] : t[j];
#pragma unroll
    for (int j = 0; j < 2; ++j) t[j] = (i & 2) ? t[j + 2] : t[j];
    return (i & 1) ? t[1] : t[0];
}

// What a slice leaves for the merge.
struct LpParts {
    float4* stats;       // [n_parts][ld]  (m, l, w, entries as int bits)
    float2* top;         // [n_parts][KC][ld]  (a, column as int bits), best first
    // [KC + 1][ld] float_key or 0.  Entry i < KC: the largest m of the slices
    // with index i modulo KC, so KC columns of the row reach the smallest of
    // them (and few others do, once every entry stands for many slices).
    // Entry KC: the largest KC-th value of any slice, which serves until then.
    uint32_t* floor;
    int ld;              // rows of the chunk buffer
};

template <int KC>
__device__ __forceinline__ void store_part(const LpParts& p, int part, int row,
                                           const RunningStats& st, const ThreadTop<KC>& tt) {
    int n = 0;
    if constexpr (KC > 0) {
        n = tt.count();
#pragma unroll
        for (int e = 0; e < KC; ++e)
            if (e < n)
                p.top[((size_t)part * KC + e) * p.ld + row] =
                    make_float2(tt.v[e], __int_as_float(tt.id[e]));
        atomicMax(&p.floor[(size_t)(part % KC) * p.ld + row], float_key(st.m));
        if (n == KC) atomicMax(&p.floor[(size_t)KC * p.ld + row], float_key(tt.v[KC - 1]));
    }
    p.stats[(size_t)part * p.ld + row] = make_float4(st.m, st.l, st.w, __int_as_float(n));
}

// A value just below the key's: columns below a row's floor cannot be among
// the KC best, columns equal to it still can (by a lower id).  Below +0 comes
// -0, which is not below it; below -inf (and for no key) nothing does.
__device__ __forceinline__ float below_key(uint32_t k) {
    if (k <= 0x007fffffu) return kNegInf;              // float_key(-inf)
    return key_float(k == 0x80000000u ? k - 2 : k - 1);
}
template <int KC>
__device__ __forceinline__ float row_floor(const LpParts& p, int row) {
    uint32_t k = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < KC; ++i) k = min(k, __ldcg(&p.floor[(size_t)i * p.ld + row]));
    return below_key(max(k, __ldcg(&p.floor[(size_t)KC * p.ld + row])));
}

// A 64-column slice from a tile of the fp32 CUDA-core GEMM.
template <int KC>
struct SimtLogprob {
    float s;                         // |s|
    float c;
    int neg;
    int64_t V;
    int rows;
    const float* bias;               // [V] fp32 or null
    LpParts parts;
    __device__ void operator()(float (*C)[kSimtTile + 1], int m0, int64_t n0, int nt) const {
        const int r = threadIdx.x;
        if (r >= kSimtTile || m0 + r >= rows) return;
        const int ncols = (int)((V - n0) < kSimtTile ? (V - n0) : kSimtTile);
        RunningStats rs;
        ThreadTop<KC> tt;
        if constexpr (KC > 0) tt.init(row_floor<KC>(parts, m0 + r));
        float mx = -CUDART_INF_F;
        for (int i = 0; i < ncols; ++i) {
            float a = C[r][i] + (bias != nullptr ? bias[n0 + i] : 0.f);
            if (neg) a = -a;
            C[r][i] = a;
            mx = fmaxf(mx, a);
            if constexpr (KC > 0)
                if (a > tt.v[KC - 1]) tt.insert(a, (int)n0 + i);
        }
        // l by e^(s (a - m)), not 2^(c (a - m)): c's rounding alone would move a
        // term 15 below the maximum by 1e-6 of itself; summed in fp64, so that
        // small terms after a large one are not cut 64 times
        const float ref = mx == -CUDART_INF_F ? 0.f : mx;
        double l = 0.0, w = 0.0;
        for (int i = 0; i < ncols; ++i) {
            const float d = C[r][i] - ref;
            const float e = expf(d * s);
            l += (double)e;
            w += (double)(e * fmaxf(d * c, -1e4f));            // (a NaN is in e)
        }
        rs.m = mx;
        rs.l = (float)l;
        rs.w = (float)w;
        store_part<KC>(parts, nt, m0 + r, rs, tt);
    }
};

// (value, id) as one integer that is larger for what ranks first: the larger
// value, then the lower id (0 to 2^31 - 1).  0 stands for nothing.
__device__ __forceinline__ uint64_t rank_key(float v, int id) {
    return (uint64_t)float_key(v) << 32 | (uint32_t)(0x7fffffff - id);
}
__device__ __forceinline__ float rank_value(uint64_t k) { return key_float((uint32_t)(k >> 32)); }
__device__ __forceinline__ int rank_id(uint64_t k) { return 0x7fffffff - (int)(uint32_t)k; }

// This lane and lane ^ d exchange: keep the larger key if `larger`.
__device__ __forceinline__ uint64_t warp_exchange(uint64_t k, int d, bool larger) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, k, d);
    return (k > o) == larger ? k : o;
}

// The 32 best of a sorted list (lane j the j-th) and 32 offers, sorted: sort
// the offers, best first; max(list[i], offers[31 - i]) are the 32 best, and a
// bitonic sequence.  (Not inlined: it is used in unrolled loops.)
__device__ __noinline__ uint64_t warp_merge_best(uint64_t list, uint64_t k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1)
            k = warp_exchange(k, d, ((lane & size) == 0) == ((lane & d) == 0));
    const uint64_t r = __shfl_sync(0xffffffffu, k, 31 - lane);
    list = list > r ? list : r;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) list = warp_exchange(list, d, (lane & d) == 0);
    return list;
}

// ======================================================================
// Candidate list of one row held across a warp: lane j has the j-th best
// key, of which the first KC count (0: none yet).
// ======================================================================
template <int KC>
struct WarpTop {
    uint64_t key = 0;

    // Every lane offers one (x, col); x = -inf (or NaN) offers nothing.  A few
    // that enter are inserted one by one (about 100 cycles each); more are
    // sorted, and merged with the list, by bitonic steps (about 700 cycles).
    __device__ __forceinline__ void offer(float x, int col, int lane) {
        offer_key(x > kNegInf ? rank_key(x, col) : 0, lane);
    }
    __device__ __forceinline__ void offer_key(uint64_t k, int lane) {
        uint32_t mask = __ballot_sync(0xffffffffu, k > __shfl_sync(0xffffffffu, key, KC - 1));
        if (__popc(mask) > 6) {
            key = warp_merge_best(key, k, lane);
            return;
        }
        while (mask != 0) {
            const int src = __ffs(mask) - 1;
            mask &= mask - 1;
            const uint64_t x1 = __shfl_sync(0xffffffffu, k, src);
            const int pos = __popc(__ballot_sync(0xffffffffu, key > x1));   // a prefix of lanes
            const uint64_t up = __shfl_up_sync(0xffffffffu, key, 1);
            key = lane > pos ? up : (lane == pos ? x1 : key);
        }
    }
};

// ---------------------------------------------------------------- exact dot products
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The weight of a head, whole (row-major, T = bf16 or fp32) or in 4 bits
// (group > 0: two nibbles a byte, element 2i low, and a bf16 scale for each
// group of a row).
struct HeadWeight {
    const void* W;
    const __nv_bfloat16* scales;     // [V][groups]
    int group;
    int groups;
};

__device__ __forceinline__ int nibble(uint32_t w, int i) {
    return ((int)(w << (28 - 4 * i))) >> 28;       // two's complement
}

constexpr int kDots = 4;             // rows of W per group of dot products

// This thread's share of <x, W_v[j]>, j < kDots, v[j] < 0 being skipped; the
// block's threads share a row, and four rows' loads are in flight together.
// Products of two bf16 (and of 4-bit values) are exact in fp32; products of
// fp32 are taken in fp64; the sums are in fp64.
template <class T>
__device__ __forceinline__ void dot_share(const T* __restrict__ x, const HeadWeight& hw,
                                          const int (&v)[kDots], int64_t D, int tid, int threads,
                                          double (&z)[kDots]) {
#pragma unroll
    for (int j = 0; j < kDots; ++j) z[j] = 0.0;
    if constexpr (sizeof(T) == 2) {
        const uint4* xq = reinterpret_cast<const uint4*>(x);
        const int n = (int)(D / 8);
        if (hw.group > 0) {
            for (int i = tid; i < n; i += threads) {
                float f[8];
                unpack8(__ldg(xq + i), f);
                const int gi = (8 * i) / hw.group;
                uint32_t w[kDots] = {};
                float c[kDots] = {};
#pragma unroll
                for (int j = 0; j < kDots; ++j)
                    if (v[j] >= 0) {
                        w[j] = __ldg(static_cast<const uint32_t*>(hw.W) + (int64_t)v[j] * n + i);
                        c[j] = __bfloat162float(hw.scales[(int64_t)v[j] * hw.groups + gi]);
                    }
#pragma unroll
                for (int j = 0; j < kDots; ++j) {
                    if (v[j] < 0) continue;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        z[j] += (double)(f[k] * ((float)nibble(w[j], k) * c[j]));
                }
            }
        } else {
            for (int i = tid; i < n; i += threads) {
                float f[8];
                unpack8(__ldg(xq + i), f);
                uint4 w[kDots] = {};
#pragma unroll
                for (int j = 0; j < kDots; ++j)
                    if (v[j] >= 0)
                        w[j] = __ldg(reinterpret_cast<const uint4*>(hw.W) + (int64_t)v[j] * n + i);
#pragma unroll
                for (int j = 0; j < kDots; ++j) {
                    if (v[j] < 0) continue;
                    float g[8];
                    unpack8(w[j], g);
#pragma unroll
                    for (int k = 0; k < 8; ++k) z[j] += (double)(f[k] * g[k]);
                }
            }
        }
    } else {
        for (int64_t i = tid; i < D; i += threads) {
            const double xi = (double)x[i];
#pragma unroll
            for (int j = 0; j < kDots; ++j) {
                if (v[j] < 0) continue;
                z[j] += xi * (double)__ldg(static_cast<const float*>(hw.W) + (int64_t)v[j] * D + i);
            }
        }
    }
}

// dst[0, n) = src[0, n_src) and zeros after it, in 16-byte vectors.
__global__ void k_pad_rows(const uint4* __restrict__ src, int64_t n_src, uint4* __restrict__ dst,
                           int64_t n) {
    const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (i < n) dst[i] = i < n_src ? src[i] : make_uint4(0, 0, 0, 0);
}

struct LpMergeParams {
    LpParts parts;
    int n_parts;
    int64_t D, V, ignore_index;
    float s, c;
    const void* H;                   // chunk's hidden states [rows, D]
    HeadWeight hw;
    const void* bias;                // [V] (type of H) or null
    const int64_t* token;            // chunk's tokens or null
    int k;
    float* logprob;                  // chunk's outputs, each may be null
    float* entropy;
    float* lse;
    float* lse_lo;                   // what rounding took off lse, or null
    int32_t* top_ids;                // [rows][k]
    float* top_logprobs;             // [rows][k]
    int32_t* n_err;                  // counts tokens outside [0, V), or null
    const int32_t* dev_err;          // the sweep's device error bits, or null
};

constexpr int kMergeKeep = 6;        // slices a thread keeps in registers

__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = (uint32_t)(k >> 32);
    const uint32_t m = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == m ? (uint32_t)k : 0u);
    return (uint64_t)m << 32 | lo;
}

// The KC largest of a warp's keys, n per lane; lane r gets the r-th (0: there
// are fewer).  Keys are distinct, and used up.
template <int KC, int n>
__device__ __forceinline__ uint64_t warp_draw(uint64_t (&key)[n], int lane) {
    uint64_t out = 0;
    for (int r = 0; r < KC; ++r) {
        uint64_t best = key[0];
#pragma unroll
        for (int j = 1; j < n; ++j) best = key[j] > best ? key[j] : best;
        best = warp_max(best);
        if (best == 0) break;
#pragma unroll
        for (int j = 0; j < n; ++j) key[j] = key[j] == best ? 0 : key[j];
        out = lane == r ? best : out;
    }
    return out;
}

// One block per row.
//
// Statistics: two passes over the slices' (m, l, w), the second in fp64.
//
// Candidates: a slice's m is its best column's value, so the KC best columns
// lie in the KC slices that rank first by m (ties: by slice, which is by
// column), and of the r-th of them only the first KC - r entries matter.
// Warps draw the slices, then the columns, by warp-wide maxima.
//
// Dot products in fp64: the given token and all KC candidates, and the result
// sorted by them.  (A candidate past the k-th may be any distance below it in
// fp32 and still be the best, where its products cancel: how far off fp32 is
// shows only in sum |x_i w_i|, which takes the same loads.)
//
// Four warps share a group of dot products.  With few rows a block has four
// such sets (THREADS = 512): the latency of one row is the kernel's (one token
// of 2048 x 32000 with 8 alternatives: 41 us a call, 47 with one set).  With
// many rows one set (128) leaves room for more rows per SM (4096 tokens of
// 2560 x 151936: 2.84 ms, 2.94 with four).
template <int KC, class T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_logprob_merge(const LpMergeParams p) {
    constexpr int NW = 4;                              // warps that read and draw the slices
    constexpr int SETS = THREADS / 128;
    constexpr int KA = KC == 0 ? 1 : KC;
    constexpr int CHUNK = kMergeKeep * 32 * NW;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ float sm_max[NW];
    __shared__ double sm_l[NW], sm_w[NW];
    __shared__ uint64_t head_key[NW * 32];
    __shared__ int sel_part[KA], sel_n[KA];
    __shared__ uint64_t ent_key[KA * KA];
    __shared__ float cand_v[KA];
    __shared__ int cand_id[KA];
    __shared__ double cand_z[KA + 1];                  // the given token's last
    __shared__ double sm_z[4][KA + 1];
    const float4* stats = p.parts.stats + row;
    const size_t ld = p.parts.ld;
    // launched while the kernel before may still run: wait for its results
    // (returns at once after an ordinary launch)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.dev_err != nullptr && *p.dev_err != 0) {
        // a wait of the sweep ran out: some slices were never written
        if (tid == 0) {
            if (p.logprob != nullptr) p.logprob[row] = CUDART_NAN_F;
            if (p.entropy != nullptr) p.entropy[row] = CUDART_NAN_F;
            if (p.lse != nullptr) p.lse[row] = CUDART_NAN_F;
            if (p.lse_lo != nullptr) p.lse_lo[row] = 0.f;
        }
        if (KC > 0 && tid < p.k) {
            p.top_ids[(size_t)row * p.k + tid] = -1;
            p.top_logprobs[(size_t)row * p.k + tid] = CUDART_NAN_F;
        }
        return;
    }

    // ---- statistics: a thread's first slices stay in registers between passes
    float4 kept[kMergeKeep];
    float mx = kNegInf;
    auto load_chunk = [&](int c0) {
#pragma unroll
        for (int j = 0; j < kMergeKeep; ++j) {
            const int k = c0 + tid + j * 32 * NW;
            kept[j] = warp < NW && k < p.n_parts ? stats[k * ld] : make_float4(kNegInf, 0.f, 0.f, 0.f);
        }
    };
    load_chunk(0);
#pragma unroll
    for (int j = 0; j < kMergeKeep; ++j) mx = fmaxf(mx, kept[j].x);
    if (warp < NW)
        for (int k = tid + CHUNK; k < p.n_parts; k += 32 * NW) mx = fmaxf(mx, stats[k * ld].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (warp < NW && lane == 0) sm_max[warp] = mx;
    if (tid < KC) {
        sel_n[tid] = 0;
        cand_id[tid] = -1;
        cand_v[tid] = kNegInf;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) mx = fmaxf(mx, sm_max[i]);
    double l = 0.0, w = 0.0;
    // Slices below the row's floor hold none of the KC best.
    float floor = kNegInf;
    if (KC > 0 && p.parts.floor != nullptr) {
        const uint32_t k = lane <= KC ? p.parts.floor[(size_t)lane * ld + row] : 0u;
        const uint32_t least = __reduce_min_sync(0xffffffffu, lane < KC ? k : 0xffffffffu);
        floor = below_key(max(least, __shfl_sync(0xffffffffu, k, KC)));
    }
    uint64_t drawn = 0;                                // lane r: the warp's r-th slice so far
    for (int c0 = 0; warp < NW && c0 < p.n_parts; c0 += CHUNK) {
        if (c0 > 0) load_chunk(c0);
        uint64_t key[kMergeKeep + 1];
#pragma unroll
        for (int j = 0; j < kMergeKeep; ++j) {
            const float4 s = kept[j];
            if (s.x != kNegInf || s.y != 0.f) {        // a slice with a logit (or a NaN)
                const float d = s.x - mx;
                const double f = (double)expf(d * fabsf(p.s));
                l += f * s.y;
                w += f * ((double)s.z + (double)fmaxf(d * p.c, -1e4f) * s.y);
            }
            key[j] = s.x > floor && __float_as_int(s.w) > 0
                         ? rank_key(s.x, c0 + tid + j * 32 * NW) : 0;
        }
        key[kMergeKeep] = drawn;
        if constexpr (KC > 0) drawn = warp_draw<KC, kMergeKeep + 1>(key, lane);
    }
    l = warp_sum(l);
    w = warp_sum(w);
    if (warp < NW) {
        if (lane == 0) { sm_l[warp] = l; sm_w[warp] = w; }
        head_key[tid] = drawn;
    }
    __syncthreads();

    // ---- candidates
    if constexpr (KC > 0) {
        if (warp == 0) {
            uint64_t key[NW];
#pragma unroll
            for (int j = 0; j < NW; ++j) key[j] = head_key[lane + 32 * j];
            const uint64_t k = warp_draw<KC, NW>(key, lane);
            if (lane < KC && k != 0) {
                sel_part[lane] = rank_id(k);
                sel_n[lane] = min(KC - lane, __float_as_int(stats[rank_id(k) * ld].w));
            }
        }
        __syncthreads();
        for (int i = tid; i < KC * KC; i += THREADS) {
            const int r = i / KC, e = i - r * KC;
            if (e >= sel_n[r]) continue;
            const float2 t = p.parts.top[((size_t)sel_part[r] * KC + e) * ld + row];
            const int id = __float_as_int(t.y);
            ent_key[i] = id >= 0 && id < p.V ? rank_key(t.x, id) : 0;
        }
        __syncthreads();
        if (warp == 0) {
            // lane r walks the r-th slice's list
            const int n = lane < KC ? sel_n[lane] : 0;
            int e = 0;
            uint64_t key = n > 0 ? ent_key[lane * KC] : 0;
            for (int r = 0; r < KC; ++r) {
                const uint64_t best = warp_max(key);
                if (best == 0) break;
                if (key == best) {
                    cand_v[r] = rank_value(best);
                    cand_id[r] = rank_id(best);
                    ++e;
                    key = e < n ? ent_key[lane * KC + e] : 0;
                }
            }
        }
    }
    int64_t y = -1;
    if (p.token != nullptr) {
        const int64_t t = p.token[row];
        if (t != p.ignore_index) {
            if (t >= 0 && t < p.V) y = t;
            else if (tid == 0 && p.n_err != nullptr) atomicAdd(p.n_err, 1);
        }
    }
    __syncthreads();

    // ---- dot products
    const T* x = static_cast<const T*>(p.H) + (int64_t)row * p.D;
    const int set = warp >> 2;
    // kDots slots by the four warps of a set; slot KC is the given token
    auto dots = [&](const int (&slot)[kDots], const int (&v)[kDots]) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < kDots; ++j) any = any || v[j] >= 0;
        if (!any) return;                              // the same for the whole set
        double z[kDots];
        dot_share<T>(x, p.hw, v, p.D, tid & 127, 128, z);
#pragma unroll
        for (int j = 0; j < kDots; ++j) {
            if (v[j] < 0) continue;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z[j] += __shfl_xor_sync(0xffffffffu, z[j], o);
            if (lane == 0) sm_z[warp & 3][slot[j]] = z[j];
        }
    };
    // after a barrier: the logit of a slot that dots() was given
    auto finish = [&](int slot, int v) {
        float b = 0.f;
        if (p.bias != nullptr) {
            if constexpr (sizeof(T) == 2)
                b = __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[v]);
            else
                b = static_cast<const float*>(p.bias)[v];
        }
        const double z = (sm_z[0][slot] + sm_z[1][slot]) + (sm_z[2][slot] + sm_z[3][slot]);
        cand_z[slot] = (double)p.s * (z + (double)b);
    };
    // the slots of the candidates, and the given token's after them
    for (int i = set * kDots; i <= KC; i += SETS * kDots) {
        int slot[kDots], v[kDots];
#pragma unroll
        for (int j = 0; j < kDots; ++j) {
            slot[j] = i + j;
            v[j] = i + j > KC ? -1 : (i + j == KC ? (int)y : cand_id[i + j]);
        }
        dots(slot, v);
    }
    __syncthreads();
    if (tid <= KC) {
        const int v = tid == KC ? (int)y : cand_id[tid];
        if (v >= 0) finish(tid, v);
    }
    __syncthreads();
    if (warp != 0) return;

    // ---- results
    l = sm_l[0];
    w = sm_w[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) { l += sm_l[i]; w += sm_w[i]; }
    // every logit -inf: lse = -inf, no information in the row
    const bool none = mx == kNegInf && l == 0.0;
    const double sm = (double)fabsf(p.s) * (double)mx;
    const double lnl = none ? 0.0 : log(l);
    const double lse = none ? -CUDART_INF : sm + lnl;
    // What logarithms of probabilities are taken against: the candidates are
    // most of a peaked row, and their logits are known exactly now, so their
    // terms of the sum are replaced.  (A log-probability near 0 is then off like
    // the rest of the row, not like fp32's lse.  lse itself and the entropy stay
    // what they are without alternatives.)
    double lse_z = lse;
    if constexpr (KC > 0) {
        double dl = 0.0;
        if (lane < KC && cand_id[lane] >= 0) {
            const double t = cand_z[lane] - sm;
            const double t0 = (double)fabsf(p.s) * ((double)cand_v[lane] - (double)mx);
            if (fabs(t - t0) <= 1.0) dl = exp(t) - exp(t0);        // (not at infinities)
        }
        dl = warp_sum(dl);
        if (!none && dl != 0.0) lse_z = sm + log(l + dl);
    }
    if (lane == 0) {
        if (p.lse != nullptr) p.lse[row] = (float)lse;
        if (p.lse_lo != nullptr)
            p.lse_lo[row] = isfinite((float)lse) ? (float)(lse - (double)(float)lse) : 0.f;
        if (p.entropy != nullptr)
            p.entropy[row] = none ? 0.f : (float)(lnl - 0.69314718055994530942 * (w / l));
        if (p.logprob != nullptr)
            p.logprob[row] = y < 0 ? 0.f : (none ? kNegInf : (float)(cand_z[KC] - lse_z));
    }
    if constexpr (KC > 0) {
        const int id = lane < KC ? cand_id[lane] : -1;
        // (a NaN ranks last: every rank is taken once, every output written)
        auto value = [&](int j) { return cand_z[j] == cand_z[j] ? cand_z[j] : -CUDART_INF; };
        const double z = id >= 0 ? value(lane) : -CUDART_INF;
        int rank = 0;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
            const int ij = cand_id[j];
            const double zj = value(j);
            if (ij >= 0 && (zj > z || (zj == z && ij < id))) ++rank;
        }
        const int found = __popc(__ballot_sync(0xffffffffu, id >= 0));
        if (id >= 0 && rank < p.k) {
            p.top_ids[(size_t)row * p.k + rank] = id;
            p.top_logprobs[(size_t)row * p.k + rank] = (float)(z - lse_z);
        }
        if (lane >= found && lane < p.k) {             // fewer logits above -inf than asked for
            p.top_ids[(size_t)row * p.k + lane] = -1;
            p.top_logprobs[(size_t)row * p.k + lane] = lse == lse ? kNegInf : CUDART_NAN_F;
        }
    }
}

// ======================================================================
// Gradient.  For upstream a = d/d logprob (0 where the token is ignored) and
// e = d/d entropy:
//   G_v = s ( p_v (-(a + e entropy) - e log p_v) + a [v = y] ).
// With q = acc c' - lse log2(e) = log2 p_v:  G_v = 2^q (kap - ee q) + ta [v = y].
// In fp32, whose results show the rounding of lse log2(e) (2^-20 of p at a lse
// of 16): with r = lse / s rounded and t = s r - lse,
//   q = s (acc - r) + t = ln p_v,   G_v = e^q (kap - ee q) + ta [v = y].
// ======================================================================
struct LpCoef {
    float* lse2;         // [chunk]; fp32: r
    float* kap;
    float* ee;
    float* ta;
    int32_t* y;          // validated token or -1
    // What rounding to bf16 took off G at the token's column (set by the
    // sweep): that element is most of a row, and its rounding would be as
    // large an error as the rounding of the results.  dH, dW and db get it
    // back; for dW a column's tokens are chained in increasing order.  (Not
    // where G has two terms.)
    float* res;          // (fp32: t instead)
    int32_t* first;      // [V] first token whose target this is (set by the sweep), or huge
    int32_t* next;       // [chunk] next token with this token's target, or rows
};

__global__ void k_logprob_coef(const int64_t* __restrict__ token, const float* __restrict__ lse,
                               const float* __restrict__ entropy, const float* __restrict__ dlp,
                               const float* __restrict__ dent, int rows, int64_t V,
                               int64_t ignore_index, float s, LpCoef o, int32_t* n_err,
                               const uint4* __restrict__ src, int64_t n_src,
                               uint4* __restrict__ dst, int64_t n_dst, int copies, bool fp32,
                               const float* __restrict__ lse_lo,
                               int32_t* dev_err, int32_t dev_err_init) {
    const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (i == 0 && dev_err != nullptr) *dev_err = dev_err_init;   // the call's first chunk
    // the padded copy of the hidden states, where they need one (see
    // pads_rows), or both copies that a G in two terms is multiplied by
    if (i < n_dst)
        dst[i] = i < n_src ? src[i] : (i < copies * n_src ? src[i - n_src] : make_uint4(0, 0, 0, 0));
    if (o.first != nullptr) {
        if (i < V) o.first[i] = 0x7fffffff;
        // a warp for every token looks for the next one of the same target
        const int64_t n = i >> 5;
        if (n < rows && token != nullptr) {
            const int64_t t = token[n];
            const int lane = (int)(i & 31);
            int64_t found = rows;
            for (int64_t b = n + 1; b < rows; b += 128) {
                unsigned hit[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t j = b + 32 * q + lane;
                    hit[q] = __ballot_sync(0xffffffffu, j < rows && token[j] == t);
                }
#pragma unroll
                for (int q = 3; q >= 0; --q)
                    if (hit[q] != 0) found = b + 32 * q + __ffs(hit[q]) - 1;
                if (found < rows) break;
            }
            if (lane == 0) o.next[n] = (int32_t)found;
        }
    }
    if (i >= rows) return;
    int64_t y = token != nullptr ? token[i] : ignore_index;
    if (y != ignore_index && (y < 0 || y >= V)) {
        if (n_err != nullptr) atomicAdd(n_err, 1);
        y = ignore_index;
    }
    const bool has = y != ignore_index;
    const float L = lse[i];
    // Every entry masked, by -inf or by a large negative value: from 2^23 on a
    // unit of fp32's last place of lse is 1 or more, and 2^(z - lse) anything up
    // to NaN.  Nothing to move.
    const bool none = L < -8388608.f;
    const float a = has && dlp != nullptr && !none ? dlp[i] : 0.f;
    const float e = dent != nullptr && !none ? dent[i] : 0.f;
    // (kap = ee = ta = 0 where there is none)
    if (fp32) {
        const double Ld = (double)L + (lse_lo != nullptr ? (double)lse_lo[i] : 0.0);
        const float r = none ? 0.f : (float)(Ld / s);
        o.lse2[i] = r;
        o.res[i] = none ? 0.f : (float)((double)r * s - Ld);
    } else {
        o.lse2[i] = none ? 0.f : L * 1.4426950408889634f;
        o.res[i] = 0.f;
    }
    o.kap[i] = e == 0.f ? -s * a : -s * fmaf(e, entropy[i], a);
    o.ee[i] = fp32 ? s * e : s * e * 0.69314718055994530942f;
    o.ta[i] = s * a;
    o.y[i] = has ? (int32_t)y : -1;
}

// What the tokens of a target from the second on give back to its row of dW:
// the sum of res[n] H[n] in fp32 and in the tokens' order, in row y (by_row)
// or the second token's row of `sum`, eight columns a thread.  A block looks
// for the first tokens of targets among every gridDim.x-th token (they are
// frequent at the chunk's begin).
//
// A link to the next token costs a load's latency, so where it is near, the
// block looks through the next 1024 tokens at once instead, and adds the rows
// it finds with 16 loads in flight (1001 tokens that share one target of
// 32000 x 2048, backward to dW: 579 us with links alone, 430 to 500 with
// windows).
constexpr int kRepeatWindow = 1024;
constexpr int kRepeatNear = 256;
__global__ void __launch_bounds__(128)
k_logprob_repeats(LpCoef k, int rows, const __nv_bfloat16* __restrict__ H, int64_t D, bool by_row,
                  float* __restrict__ sum) {
    __shared__ int list[kRepeatWindow];
    __shared__ uint32_t found[kRepeatWindow / 32];
    __shared__ int second[128], heads;
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t d = 8 * ((int64_t)blockIdx.y * blockDim.x + tid);
    for (int64_t b = blockIdx.x; b < rows; b += 128 * (int64_t)gridDim.x) {
        if (tid == 0) heads = 0;
        __syncthreads();
        const int64_t c = b + tid * (int64_t)gridDim.x;
        if (c < rows) {
            const int yc = k.y[c], nc = k.next[c];
            if (yc >= 0 && nc < rows && k.first[yc] == c) second[atomicAdd(&heads, 1)] = nc;
        }
        __syncthreads();
        const int count = heads;
        for (int s = 0; s < count; ++s) {
            float a[8] = {};
            int n = second[s];
            const int y = k.y[n];
            float* const out = sum + (int64_t)(by_row ? y : n) * D + d;
            while (n < rows) {
                const int next = k.next[n];
                int size = 1;
                __syncthreads();                       // the list is free again
                if (next - n >= kRepeatNear || next >= rows) {
                    if (tid == 0) list[0] = n;
                    __syncthreads();
                    n = next;
                } else {
                    // tokens n + 128 i + tid: bit `lane` of word 4 i + warp
#pragma unroll
                    for (int i = 0; i < kRepeatWindow / 128; ++i) {
                        const int64_t t = (int64_t)n + 128 * i + tid;
                        const uint32_t bits = __ballot_sync(0xffffffffu, t < rows && k.y[t] == y);
                        if (lane == 0) found[4 * i + (tid >> 5)] = bits;
                    }
                    __syncthreads();
                    // lane i of every warp: words 0 .. i
                    const uint32_t word = found[lane];
                    int upto = __popc(word);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += v;
                    }
                    size = __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
                    for (int i = 0; i < kRepeatWindow / 128; ++i) {
                        const int w = 4 * i + (tid >> 5);
                        const uint32_t bits = __shfl_sync(0xffffffffu, word, w);
                        const int before = __shfl_sync(0xffffffffu, upto, w) - __popc(bits);
                        if (bits >> lane & 1u)
                            list[before + __popc(bits & ((1u << lane) - 1u))] = n + 32 * w + lane;
                    }
                    __syncthreads();
                    n = k.next[list[size - 1]];
                }
                if (d >= D) continue;
                for (int j = 0; j < size; j += 16) {
                    float e[16];
                    uint4 x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const bool is = j + i < size;
                        const int64_t t = is ? list[j + i] : 0;
                        e[i] = is ? __ldg(k.res + t) : 0.f;
                        x[i] = is ? __ldg(reinterpret_cast<const uint4*>(H + t * D + d))
                                  : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (e[i] == 0.f) continue;
                        float f[8];
                        unpack8(x[i], f);
#pragma unroll
                        for (int q = 0; q < 8; ++q) a[q] = fmaf(e[i], f[q], a[q]);
                    }
                }
            }
            if (d >= D) continue;
            reinterpret_cast<float4*>(out)[0] = make_float4(a[0], a[1], a[2], a[3]);
            reinterpret_cast<float4*>(out)[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
        __syncthreads();
    }
}

// Column sums of the bf16 G [rows, Vpad] over one segment of rows (in row
// order): part[segment][V], four columns a thread, 16 rows' loads in flight.
__global__ void __launch_bounds__(128)
k_logprob_colsum(const __nv_bfloat16* __restrict__ G, int64_t ldg, int rows, int64_t V,
                 int seg_rows, float* __restrict__ part) {
    const int64_t v = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
    if (v >= V) return;
    const int r0 = blockIdx.y * seg_rows;
    const int r1 = min(rows, r0 + seg_rows);
    float a[4] = {};
#pragma unroll 16
    for (int r = r0; r < r1; ++r) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(G + (size_t)r * ldg + v));
        a[0] += __uint_as_float(w.x << 16);
        a[1] += __uint_as_float(w.x & 0xffff0000u);
        a[2] += __uint_as_float(w.y << 16);
        a[3] += __uint_as_float(w.y & 0xffff0000u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (v + i < V) part[(size_t)blockIdx.y * V + v + i] = a[i];
}

// db of one chunk: the column sums' partials (in segment order), what rounding
// took off G at the chunk's tokens (in token order), and the chunks before.
// The last chunk writes db (out), added to with `add_out`; others acc.
__global__ void k_logprob_db(const float* __restrict__ part, int nseg, int64_t V,
                             const int32_t* __restrict__ y, const float* __restrict__ res, int rows,
                             float* __restrict__ acc, int add_acc, void* out, int to_bf16,
                             int add_out) {
    __shared__ __align__(16) int32_t sy[256];
    __shared__ float sr[256];
    const int64_t v = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    float s = 0.f;
    if (v < V)
        for (int k = 0; k < nseg; ++k) s += part[(size_t)k * V + v];
    for (int r0 = 0; r0 < rows; r0 += 256) {
        __syncthreads();
        const int r = r0 + threadIdx.x;
        sy[threadIdx.x] = r < rows ? y[r] : -1;
        sr[threadIdx.x] = r < rows ? res[r] : 0.f;
        __syncthreads();
        const int n = min(256, rows - r0);
#pragma unroll 4
        for (int i = 0; i < n; i += 4) {
            const int4 q = *reinterpret_cast<const int4*>(sy + i);
            if (q.x == v || q.y == v || q.z == v || q.w == v)         // seldom
                for (int j = 0; j < 4; ++j)
                    if (sy[i + j] == v) s += sr[i + j];
        }
    }
    if (v >= V) return;
    if (add_acc) s += acc[v];
    if (out == nullptr) {
        acc[v] = s;
    } else if (to_bf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out);
        o[v] = __float2bfloat16_rn(add_out ? __bfloat162float(o[v]) + s : s);
    } else {
        float* o = static_cast<float*>(out);
        o[v] = add_out ? o[v] + s : s;
    }
}

// After a gradient: where a wait of its kernels ran out, tiles were never
// written or are partial sums, and all of it becomes NaN (bits of ones).
__global__ void k_logprob_void(const int32_t* __restrict__ dev_err, uint4* dH, int64_t nH, uint4* dW,
                               int64_t nW, uint16_t* db, int64_t nb) {
    if (*dev_err == 0) return;
    const int64_t i0 = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const uint4 ones = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (int64_t i = i0; i < nH; i += step) dH[i] = ones;
    for (int64_t i = i0; i < nW; i += step) dW[i] = ones;
    for (int64_t i = i0; i < nb; i += step) db[i] = 0xffff;
}

// What rounding x to bf16 takes off it (nothing where either is no number).
__device__ __forceinline__ float bf16_rest(float x) {
    const float r = x - __bfloat162float(__float2bfloat16_rn(x));
    return fabsf(r) < CUDART_INF_F ? r : 0.f;
}

// One element: q = log2 p.  A row without upstream gradient is exactly 0.
__device__ __forceinline__ float lp_grad(float q, float kap, float ee) {
    q = q < -1e4f ? -1e4f : q;                     // a logit of -inf: p = 0, not 0 * inf
    return ex2(q) * fmaf(-ee, q, kap);
}

struct LogprobGEpi {
    struct Params {
        CUtensorMap gmap;            // G [rows, V] bf16, box 64 x 32, 128B swizzle
        float c;                     // s log2(e)
        int64_t V;
        int rows;
        LpCoef k;
        const __nv_bfloat16* bias;   // [V] or null
    };

    // G is rounded once to bf16, the operand type of the dH and dW products.
    template <class Cfg>
    static __device__ __forceinline__ void run(const Params& p, const TileCtx& t,
                                               const AccRow& acc, Stager& st) {
        static_assert(Cfg::NSUB == 1, "one 256-column MMA per vocabulary tile");
        const int64_t n0 = t.col0;
        const int m = t.row0 + t.row;
        float L2 = 0.f, kap = 0.f, ee = 0.f, ta = 0.f;
        int yrel = -1;
        if (m < p.rows) {
            L2 = p.k.lse2[m];
            kap = p.k.kap[m];
            ee = p.k.ee[m];
            ta = p.k.ta[m];
            const int y = p.k.y[m];
            if (y >= n0 && y < n0 + Cfg::BN) yrel = (int)(y - n0);
        }
        const bool dead = kap == 0.f && ee == 0.f && ta == 0.f;
        const int ncols = (int)((p.V - n0) < Cfg::BN ? (p.V - n0) : Cfg::BN);
        const float c = p.c;
        for_each_chunk<Cfg::NCHUNK>(acc, [&](const uint32_t (&r)[32], int j) {
            float g[32];
            if (p.bias != nullptr) {
                float b[32];
                load_bias32(p.bias, n0 + 32 * j, p.V, b);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    g[i] = lp_grad(fmaf(__uint_as_float(r[i]) + b[i], c, -L2), kap, ee);
            } else {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float q0, q1, k0, k1;
                    fma2(q0, q1, __uint_as_float(r[i]), __uint_as_float(r[i + 1]), c, c, -L2, -L2);
                    fma2(k0, k1, q0, q1, -ee, -ee, kap, kap);
                    mul2(g[i], g[i + 1], k0, k1, ex2(q0), ex2(q1));
                }
            }
            if ((unsigned)(yrel - 32 * j) < 32u) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i == yrel - 32 * j) {
                        g[i] += ta;
                        p.k.res[m] = dead ? 0.f : bf16_rest(g[i]);
                        if (p.k.first != nullptr) atomicMin(p.k.first + n0 + yrel, m);
                    }
            }
            if (dead) {
#pragma unroll
                for (int i = 0; i < 32; ++i) g[i] = 0.f;
            }
            if (32 * j + 32 > ncols) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (32 * j + i >= ncols) g[i] = 0.f;
            }
            if ((j & 1) == 0) st.acquire();
            stage_bf16_half(st, j, g);
            if (j & 1) st.flush(&p.gmap, (int)(n0 + 32 * (j - 1)), t.row0 + 32 * t.q, false);
        });
    }
};

struct SimtLogprobG {
    float s;
    int64_t V, ldg;
    int rows;
    LpCoef k;
    float* G;
    const float* bias;               // [V] fp32 or null
    __device__ void operator()(float (*C)[kSimtTile + 1], int m0, int64_t n0, int) const {
        for (int idx = threadIdx.x; idx < kSimtTile * kSimtTile; idx += blockDim.x) {
            const int r = idx / kSimtTile, i = idx % kSimtTile;
            const int m = m0 + r;
            const int64_t v = n0 + i;
            if (m >= rows || v >= ldg) continue;
            float g = 0.f;
            const float kap = k.kap[m], ee = k.ee[m], ta = k.ta[m];
            if (v < V && !(kap == 0.f && ee == 0.f && ta == 0.f)) {
                const float a = C[r][i] + (bias != nullptr ? bias[v] : 0.f);
                float q = fmaf(a - k.lse2[m], s, k.res[m]);
                q = q < -1e4f ? -1e4f : q;             // a logit of -inf: p = 0, not 0 * inf
                g = expf(q) * fmaf(-ee, q, kap);
                if (v == k.y[m]) g += ta;
            }
            G[(size_t)m * ldg + v] = g;
        }
    }
};

}  // namespace fldce
