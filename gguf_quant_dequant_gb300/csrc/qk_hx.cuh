// qk_hx.cuh -- activations of the tensor-core GEMVs: one unit (256 elements)
// staged by a warp and turned into its MMA's B fragments (qk_hunits.cuh).
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "qk_ptx.cuh"

namespace qk {
namespace hm {

constexpr int kXBB = 128;   // prepared bytes per x-block: 2 planes x 8 words x 8 bytes

// x -> B fragments in shared memory, one unit (256 elements, 8 x-blocks)
// at a time by the warp that uses it.  Local x-block j of the unit, plane h:
//   xb[(2j + h) * 64 + 8i] = half2(x_h[4i], x_h[4i+2]), half2(x_h[4i+1], x_h[4i+3])
// with x' = x * 2^-e, x_0 = fp16(x'), x_1 = fp16(x' - x_0); xm[j] = (sum of x
// over the block, 2^e, sum over its first 16 elements, over its last 16).
// e = 0 unless max|x| of the block reaches 2^15, then the block is scaled
// into [2^14, 2^15) (LOWEST below 0: always).  Lane l takes elements 8q .. 8q + 7 (q = l % 4) of
// local block l / 4; blocks past x are zero.
// The unit's x for lane `lane` (eight floats) copied into its 32-byte slot
// of `xs` without holding registers (cp.async; zeros past x).
__device__ __forceinline__ void load_unit_x(const float* __restrict__ x, int nxb, int u, int lane, float* xs) {
    const int j = 8 * u + (lane >> 2), q = lane & 3;
    float* d = xs + 8 * lane;
    if (j < nxb) {
        cp_async16(d, x + 32 * j + 8 * q);
        cp_async16(d + 4, x + 32 * j + 8 * q + 4);
    } else {
        *reinterpret_cast<float4*>(d) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        *reinterpret_cast<float4*>(d + 4) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
}
// The eight elements (a, b) of lane `lane`: hi and lo as four half2 each (of
// elements {0, 2}, {1, 3}, {4, 6}, {5, 7}), and the block's (sum, 2^e, sum of
// the first 16, sum of the last 16) in the block's first lane.  The exponent
// is kept at LOWEST and above: 0 leaves small blocks as they are (an absolute
// error of 2^-25), -100 scales them up too.
template <int LOWEST>
__device__ __forceinline__ float4 split_x(float4 a, float4 b, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    const float amax_a = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w)));
    float amax = fmaxf(amax_a, fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
    // The eight elements' sum by packed pair adds (any order: an fp32 block sum).
    const float2 s2 = __fadd2_rn(__fadd2_rn(make_float2(a.x, a.y), make_float2(a.z, a.w)),
                                 __fadd2_rn(make_float2(b.x, b.y), make_float2(b.z, b.w)));
    float sum = s2.x + s2.y;
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);           // sum of 16 elements (one half)
    const float other = __shfl_xor_sync(0xffffffffu, sum, 2);
    // Scale exponent: floor(log2 max|x|) - 14, or LOWEST.
    const int ex = (int)((__float_as_uint(amax) >> 23) & 255u) - 127;
    const int e = max(LOWEST, ex - 14);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
    // Words 2q and 2q+1: elements 8q + {0,2}, {1,3}, {4,6}, {5,7}; each pair
    // rounded to fp16 by one packed convert, its residual by another.
    constexpr int kPair[4][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}};
    // x' = x 2^-e on the loads' natural register pairs.
    const float2 s01 = __fmul2_rn(make_float2(a.x, a.y), make_float2(down, down));
    const float2 s23 = __fmul2_rn(make_float2(a.z, a.w), make_float2(down, down));
    const float2 s45 = __fmul2_rn(make_float2(b.x, b.y), make_float2(down, down));
    const float2 s67 = __fmul2_rn(make_float2(b.z, b.w), make_float2(down, down));
    const float xs8[8] = {s01.x, s01.y, s23.x, s23.y, s45.x, s45.y, s67.x, s67.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a0 = xs8[kPair[k][0]], b0 = xs8[kPair[k][1]];
        const __half2 h = __floats2half2_rn(a0, b0);
        const float2 hf = __half22float2(h);
        const __half2 l = __floats2half2_rn(a0 - hf.x, b0 - hf.y);   // x' - hi, exact
        hi[k] = *reinterpret_cast<const uint32_t*>(&h);
        lo[k] = *reinterpret_cast<const uint32_t*>(&l);
    }
    return make_float4(sum + other, up, sum, other);
}
template <int LOWEST = 0>
__device__ __forceinline__ void prep_unit_x(const float* xs, uint8_t* xb, float4* xm, int lane) {
    const int jl = lane >> 2, q = lane & 3;
    const float4 a = *reinterpret_cast<const float4*>(xs + 8 * lane), b = *reinterpret_cast<const float4*>(xs + 8 * lane + 4);
    uint32_t hi[4], lo[4];
    const float4 m = split_x<LOWEST>(a, b, hi, lo);
    *reinterpret_cast<uint4*>(xb + jl * kXBB + 16 * q) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(xb + jl * kXBB + 64 + 16 * q) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (q == 0) xm[jl] = m;
}

}  // namespace hm
}  // namespace qk
