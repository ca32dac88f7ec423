// qk_rows.cuh -- rows of activations by eight elements a lane, and their way
// into the blocks of the paged cache: shared by the append kernels.
#pragma once
#include <cstdint>

#include "qk_qlanes.cuh"

namespace qk {
namespace kv {

// Elements at .. at + 7 of a row, as fp32 (vec: the address is 16-byte aligned).
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t at, bool vec, float (&x)[8]) {
    if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        uint32_t w[4];
        if (vec) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float* p = static_cast<const float*>(base) + at;
        if (vec) {
            const float4 f = __ldcs(reinterpret_cast<const float4*>(p)), g = __ldcs(reinterpret_cast<const float4*>(p + 4));
            x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w, x[4] = g.x, x[5] = g.y, x[6] = g.z, x[7] = g.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = p[i];
        }
    }
}

// The lane's part of one block, e of four, at dst (nullptr: nothing is written).
template <int T>
__device__ __forceinline__ void append_block(const float (&x)[8], uint8_t* dst, int e) {
    constexpr int kOff = T == T_Q8_0 ? 0 : (T == T_Q5_0 ? 16 : 8);
    constexpr int kLo = T == T_Q8_0 ? -128 : -kOff;
    constexpr int kHi = T == T_Q8_0 ? 127 : kOff - 1;
    constexpr float kDiv = T == T_Q8_0 ? 127.0f : (T == T_Q5_0 ? 15.0f : 7.0f);
    float m = 0.0f;   // NaN elements are skipped, as the quantizer's scan does
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t db = ql::half_bits(__fdiv_rn(m, kDiv));
    const float d = ql::half_val(db);
    uint32_t q[8];
    if (d > 0.0f) {
        group_codes<8, kLo, kHi, kOff>(x, d, q);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = (uint32_t)kOff;
    }
    const uint32_t w0 = ql::bytes4(q), w1 = ql::bytes4(q + 4);
    if constexpr (T == T_Q8_0) {
        if (dst) {
            if (e == 0) ql::st_u16(dst, db);
            uint8_t* p = dst + 2 + 8 * e;
            ql::st_u16(p, w0 & 0xffffu);
            ql::st_u16(p + 2, w0 >> 16);
            ql::st_u16(p + 4, w1 & 0xffffu);
            ql::st_u16(p + 6, w1 >> 16);
        }
    } else {
        // Byte j holds element j (low nibble) and j + 16 (high): lanes 0 and
        // 1 take the high nibbles from lanes 2 and 3.
        const uint32_t h0 = __shfl_xor_sync(0xffffffffu, w0, 2), h1 = __shfl_xor_sync(0xffffffffu, w1, 2);
        uint32_t fifth = 0;
        if constexpr (T == T_Q5_0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) fifth |= ((q[i] >> 4) & 1u) << i;   // byte e of the fifth-bit word
        }
        if (dst) {
            uint8_t* qs = dst + (T == T_Q5_0 ? 6 : 2);
            if (e == 0) ql::st_u16(dst, db);
            if (T == T_Q5_0) dst[2 + e] = (uint8_t)fifth;
            if (e < 2) {
                const uint32_t n0 = (w0 & 0x0F0F0F0Fu) | ((h0 & 0x0F0F0F0Fu) << 4);
                const uint32_t n1 = (w1 & 0x0F0F0F0Fu) | ((h1 & 0x0F0F0F0Fu) << 4);
                uint8_t* p = qs + 8 * e;
                ql::st_u16(p, n0 & 0xffffu);
                ql::st_u16(p + 2, n0 >> 16);
                ql::st_u16(p + 4, n1 & 0xffffu);
                ql::st_u16(p + 6, n1 >> 16);
            }
        }
    }
}

}  // namespace kv
}  // namespace qk
