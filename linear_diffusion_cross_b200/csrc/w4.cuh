// w4.cuh -- the 4-bit head weight: quantisation and products for few tokens.
//
// W[v, d] = q[v, d] * scale[v, d / group]: q is a two's complement nibble
// (byte i of a row holds element 2i in its low half and 2i + 1 in its high
// half), scale is bf16.
#pragma once
#include "logprob.cuh"

namespace fldce {

// One warp per (row, group): scale = bf16(max |w| / 7), q = round(w / scale)
// to nearest even, clamped to [-7, 7] (the rounded scale may be a little
// below max / 7).  A group of zeros has scale 0 and q = 0.
template <class T>
__global__ void k_w4_quantize(const T* __restrict__ W, int64_t V, int64_t D, int group,
                              uint8_t* __restrict__ packed, __nv_bfloat16* __restrict__ scales) {
    const int64_t groups = (D + group - 1) / group;
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t u = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5); u < V * groups;
         u += stride) {
        const int64_t v = u / groups, gi = u - v * groups;
        const int64_t d0 = gi * group;
        const int n = (int)min((int64_t)group, D - d0);      // a multiple of 32
        const T* src = W + v * D + d0;
        float x[4], mx = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {                        // elements 64 i + 2 lane, + 1
            const int e = 64 * i + 2 * lane;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float f = 0.f;
                if (e < n) {
                    if constexpr (sizeof(T) == 2) f = __bfloat162float(src[e + k]);
                    else f = src[e + k];
                }
                x[2 * i + k] = f;
                mx = fmaxf(mx, fabsf(f));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(mx, 7.f));
        const float sc = __bfloat162float(sb);
        if (lane == 0) scales[v * groups + gi] = sb;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 64 * i + 2 * lane;
            if (e >= n) continue;
            uint32_t b = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float r = sc > 0.f ? rintf(__fdiv_rn(x[2 * i + k], sc)) : 0.f;
                const int q = (int)fminf(7.f, fmaxf(-7.f, r));
                b |= (uint32_t)(q & 15) << (4 * k);
            }
            packed[(v * D + d0 + e) / 2] = (uint8_t)b;
        }
    }
}

constexpr int kW4Tokens = 8;      // tokens per pass over the weight

// Logits of up to kW4Tokens tokens, one warp per vocabulary row.
// out[n * ldo + v] = <x_n, W_v> (+ bias[v]).
template <class OutT>
__global__ void __launch_bounds__(256)
k_w4_rows(const __nv_bfloat16* __restrict__ x, int n_tok, HeadWeight hw,
          const __nv_bfloat16* __restrict__ bias, int64_t V, int64_t D, OutT* __restrict__ out,
          int64_t ldo) {
    const int lane = threadIdx.x & 31;
    const int64_t stride = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t v = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5); v < V;
         v += stride) {
        float acc[kW4Tokens] = {};
        const uint32_t* q = reinterpret_cast<const uint32_t*>(hw.W) + v * (D / 8);
        for (int64_t i = lane; i < D / 8; i += 32) {
            const uint32_t wq = __ldg(q + i);
            const float sc = __bfloat162float(hw.scales[v * hw.groups + (8 * i) / hw.group]);
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = (float)nibble(wq, k) * sc;
#pragma unroll
            for (int n = 0; n < kW4Tokens; ++n) {
                if (n >= n_tok) break;
                const uint4 a = __ldg(reinterpret_cast<const uint4*>(x + n * D) + i);
                const uint32_t au[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 t =
                        __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&au[k]));
                    acc[n] = fmaf(f[2 * k], t.x, acc[n]);
                    acc[n] = fmaf(f[2 * k + 1], t.y, acc[n]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < kW4Tokens; ++n) {
            if (n >= n_tok) break;
            float s = acc[n];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) {
                if (bias != nullptr) s += __bfloat162float(bias[v]);
                if constexpr (sizeof(OutT) == 2) out[n * ldo + v] = __float2bfloat16_rn(s);
                else out[n * ldo + v] = s;
            }
        }
    }
}

constexpr int kLogitPart = 1024;  // columns per slice of k_logit_parts

// The slices' statistics from logits in memory: one warp per (token, slice).
// `ld` of the parts is the chunk's rows; row0 is the first token's row in it.
template <int KC>
__global__ void __launch_bounds__(128)
k_logit_parts(const float* __restrict__ logits, int64_t ldl, int n_tok, int row0, int64_t V,
              float c, int neg, LpParts parts, int n_parts) {
    const int lane = threadIdx.x & 31;
    const int64_t u = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
    if (u >= (int64_t)n_parts * n_tok) return;
    const int tok = (int)(u / n_parts), part = (int)(u - (int64_t)tok * n_parts);
    const int64_t v0 = (int64_t)part * kLogitPart;
    const float* src = logits + tok * ldl;
    RunningStats rs;
    WarpTop<KC == 0 ? 1 : KC> wt;
    for (int i = 0; i < kLogitPart; i += 32) {
        const int64_t v = v0 + i + lane;
        if (v0 + i >= V) break;
        float a = -CUDART_INF_F;
        if (v < V) a = neg ? -src[v] : src[v];
        const float ref = rs.rebase(fmaxf(rs.m, a), c);
        rs.add(a, ref, c);
        if constexpr (KC > 0) wt.offer(a, (int)v, lane);
    }
    float mx = rs.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    rs.rebase(mx, c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        rs.l += __shfl_xor_sync(0xffffffffu, rs.l, o);
        rs.w += __shfl_xor_sync(0xffffffffu, rs.w, o);
    }
    int n = 0;
    if constexpr (KC > 0) {
        const bool has = lane < KC && wt.v > -CUDART_INF_F;
        n = __popc(__ballot_sync(0xffffffffu, has));
        if (has)
            parts.top[((size_t)part * KC + lane) * parts.ld + row0 + tok] =
                make_float2(wt.v, __int_as_float(wt.id));
    }
    if (lane == 0)
        parts.stats[(size_t)part * parts.ld + row0 + tok] =
            make_float4(mx, rs.l, rs.w, __int_as_float(n));
}

}  // namespace fldce
