// w4.cuh -- quantisation of the 4-bit head weight.
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

}  // namespace fldce
