// qk_dunits.cuh -- unit decoders for several activation rows at a time: 16
// weight rows x 256 weights against NT (4 or 8) rows of x, each weight
// converted once.
//
// Arithmetic as qk_hunits.cuh: exact integer codes less an offset as fp16 A
// fragments, x as hi + lo fp16 terms after a power of two per 32-block, fp32
// sums scaled per block.  There a warp's four column groups hold four parts of
// K for one row of x; here all sixteen k of an MMA come from one 32-block and
// the eight columns are rows of x: four rows by (hi, lo), or eight rows with hi
// and lo in two MMAs.  So one MMA serves four rows instead of one, and a
// thread's sums are whole: row g and g + 8 against its own row(s) of x.
//
// Thread (g, t) supplies rows g and g + 8; of a 32-block's eight code words
// (four weights each) it takes words 2t and 2t + 1 in steps 0 and 1, or, where
// the weights are scaled by sixteens or the two halves sit in the nibbles of
// the same bytes (kW4), words t and t + 4, so that a step is one half of the
// block.  The scales of a pair of blocks are worked out by the thread whose
// group it was there (t = pair) and handed round the quad.
#pragma once
#include <cstdint>

#include "qk_hunits.cuh"
#include "qk_hx.cuh"

namespace qk {
namespace dm {
using namespace hm;

// Prepared x of one unit: NT = 4 [block][row][plane][64 bytes], NT = 8
// [block][plane][row][64 bytes] (conflict-free for the B loads); the words of a
// plane in their order, or 0, 4, 1, 5, .. (kW4).  xm [block][row]: sum, 2^e,
// sums of the halves.
template <int NT>
__device__ __forceinline__ uint32_t x_off(int blk, int row, int plane) {
    return NT == 4 ? (uint32_t)(blk * 512 + row * 128 + plane * 64) : (uint32_t)(blk * 1024 + plane * 512 + row * 64);
}
constexpr int kXRow = 8 * 128;   // bytes of a row of x in a unit
template <int NT, bool W4>
__device__ __forceinline__ void put_x(float4 a, float4 b, uint8_t* xb, float4* xm, int row, int lane) {
    const int blk = lane >> 2, q = lane & 3;
    uint32_t hi[4], lo[4];
    const float4 m = split_x<-100>(a, b, hi, lo);
    uint8_t* h = xb + x_off<NT>(blk, row, 0);
    uint8_t* l = xb + x_off<NT>(blk, row, 1);
    if constexpr (W4) {
        const int at = q < 2 ? 32 * q : 32 * (q - 2) + 8;   // words 2q and 2q + 1
        *reinterpret_cast<uint2*>(h + at) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(h + at + 16) = make_uint2(hi[2], hi[3]);
        *reinterpret_cast<uint2*>(l + at) = make_uint2(lo[0], lo[1]);
        *reinterpret_cast<uint2*>(l + at + 16) = make_uint2(lo[2], lo[3]);
    } else {
        *reinterpret_cast<uint4*>(h + 16 * q) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(l + 16 * q) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (q == 0) xm[blk * NT + row] = m;
}

// Word at a 2-byte-aligned shared address.
__device__ __forceinline__ uint32_t word_a2(const uint8_t* p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint8_t* b = reinterpret_cast<const uint8_t*>(a & ~uintptr_t(3));
    return __funnelshift_r(lds32(b), lds32(b + 4), (uint32_t)(a & 3) * 8);
}
__device__ __forceinline__ uint2 words2_a2(const uint8_t* p) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint8_t* b = reinterpret_cast<const uint8_t*>(a & ~uintptr_t(3));
    const uint32_t sh = (uint32_t)(a & 3) * 8, w0 = lds32(b), w1 = lds32(b + 4), w2 = lds32(b + 8);
    return make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh));
}
template <class V>
__device__ __forceinline__ V from(V v, int src) { return __shfl_sync(0xffffffffu, v, src); }

// Four A registers from code words of rows g and g + 8 whose codes lie under
// mask M of each byte, with the magic G and the offsets o0, o1 to add.
__device__ __forceinline__ void frag(uint32_t (&A)[4], uint32_t w0, uint32_t w1, uint32_t M, uint32_t G, uint32_t o0, uint32_t o1) {
    A[0] = hadd2(and_or(w0, M, G), o0);
    A[1] = hadd2(and_or(w1, M, G), o1);
    A[2] = hadd2(and_or(w0 >> 8, M, G), o0);
    A[3] = hadd2(and_or(w1 >> 8, M, G), o1);
}

// Scales of a block for rows g and g + 8: per half where scaled by sixteens
// (else [0] alone), and the negative residuals of the types with a min.
struct Scale {
    float f[2][2], n[2][2];   // [row][half]
};

// A decoder: UB bytes per row and unit, kW4 (above), kG16 (scaled by
// sixteens), kMin (has a residual), block(pair c, b), Ctx, load(ctx, r0, r1,
// lane), pair(ctx, c, lane, A, s): fragments A[b][step] and scales s[b] of the
// pair's two blocks.
template <int T> struct DU;

template <> struct DU<T_Q4_K> {
    static constexpr int UB = 144;
    static constexpr bool kW4 = false, kG16 = false, kMin = true;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        HU<T_Q4_K>::Row p0, p1;
        const uint8_t *r0, *r1;
    };
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane) {
        x.p0 = HU<T_Q4_K>::row_params<true>(lds128(r0), lane & 3, 15.0f);
        x.p1 = HU<T_Q4_K>::row_params<true>(lds128(r1), lane & 3, 15.0f);
        x.r0 = r0 + 16 + 8 * (lane & 3);
        x.r1 = r1 + 16 + 8 * (lane & 3);
    }
    __device__ static __forceinline__ void scales(const HU<T_Q4_K>::Row& p0, const HU<T_Q4_K>::Row& p1, int src, Scale (&s)[2]) {
        s[0].f[0][0] = from(p0.ds.x, src), s[1].f[0][0] = from(p0.ds.y, src);
        s[0].f[1][0] = from(p1.ds.x, src), s[1].f[1][0] = from(p1.ds.y, src);
        s[0].n[0][0] = from(p0.nr.x, src), s[1].n[0][0] = from(p0.nr.y, src);
        s[0].n[1][0] = from(p1.nr.x, src), s[1].n[1][0] = from(p1.nr.y, src);
    }
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c;
        const uint2 w0 = lds64(x.r0 + 32 * c), w1 = lds64(x.r1 + 32 * c);
        const uint32_t l0 = from(x.p0.clo, src), l1 = from(x.p1.clo, src), h0 = from(x.p0.chi, src), h1 = from(x.p1.chi, src);
        frag(A[0][0], w0.x, w1.x, 0x000F000Fu, 0x64006400u, l0, l1);
        frag(A[0][1], w0.y, w1.y, 0x000F000Fu, 0x64006400u, l0, l1);
        frag(A[1][0], w0.x, w1.x, 0x00F000F0u, 0x54005400u, h0, h1);
        frag(A[1][1], w0.y, w1.y, 0x00F000F0u, 0x54005400u, h0, h1);
        scales(x.p0, x.p1, src, s);
    }
};

template <> struct DU<T_Q5_K> {
    static constexpr int UB = 176;
    static constexpr bool kW4 = false, kG16 = false, kMin = true;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        HU<T_Q4_K>::Row p0, p1;
        const uint8_t *r0, *r1;
        uint2 v0, v1;   // the fifth bits of the thread's words, all blocks
    };
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane) {
        x.p0 = HU<T_Q4_K>::row_params<false>(lds128(r0), lane & 3, 31.0f);
        x.p1 = HU<T_Q4_K>::row_params<false>(lds128(r1), lane & 3, 31.0f);
        x.v0 = lds64(r0 + 16 + 8 * (lane & 3));
        x.v1 = lds64(r1 + 16 + 8 * (lane & 3));
        x.r0 = r0 + 48 + 8 * (lane & 3);
        x.r1 = r1 + 48 + 8 * (lane & 3);
    }
    __device__ static __forceinline__ uint32_t low(uint32_t w, uint32_t v, int c) { return and_or(w, 0x0F0F0F0Fu, ((v >> (2 * c)) << 4) & 0x10101010u); }
    __device__ static __forceinline__ uint32_t high(uint32_t w, uint32_t v, int c) {
        return and_or(w >> 4, 0x0F0F0F0Fu, ((v >> (2 * c)) << 3) & 0x10101010u);
    }
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c;
        const uint2 w0 = lds64(x.r0 + 32 * c), w1 = lds64(x.r1 + 32 * c);
        const uint32_t l0 = from(x.p0.clo, src), l1 = from(x.p1.clo, src), h0 = from(x.p0.chi, src), h1 = from(x.p1.chi, src);
        constexpr uint32_t M = 0x001F001Fu, G = 0x64006400u;
        frag(A[0][0], low(w0.x, x.v0.x, c), low(w1.x, x.v1.x, c), M, G, l0, l1);
        frag(A[0][1], low(w0.y, x.v0.y, c), low(w1.y, x.v1.y, c), M, G, l0, l1);
        frag(A[1][0], high(w0.x, x.v0.x, c), high(w1.x, x.v1.x, c), M, G, h0, h1);
        frag(A[1][1], high(w0.y, x.v0.y, c), high(w1.y, x.v1.y, c), M, G, h0, h1);
        DU<T_Q4_K>::scales(x.p0, x.p1, src, s);
    }
};

// Pair c: the 32-blocks (th, gl) and (th, gl + 2), th = c / 2, gl = c % 2, of
// low and high nibbles of the same bytes.
template <> struct DU<T_Q6_K> {
    static constexpr int UB = 210;
    static constexpr bool kW4 = true, kG16 = true, kMin = false;
    __device__ static __forceinline__ int block(int c, int b) { return 4 * (c >> 1) + (c & 1) + 2 * b; }
    struct Ctx {
        float f0[4], f1[4];   // d * scale of the thread's own pair: block, half
        const uint8_t *r0, *r1;
        uint32_t h0[2], h1[2];   // high bits of the current half
    };
    __device__ static __forceinline__ void own(const uint8_t* r, int t, float (&f)[4]) {
        const int at = 8 * (t >> 1) + 2 * (t & 1);
        const uint32_t u = (ld_u16(r + 192 + at) | (ld_u16(r + 196 + at) << 16)) ^ 0x80808080u;   // + 128
        const float d = h2f(ld_u16(r + 208));
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = d * (ubyte_f(u, k) - 128.0f);   // exact
    }
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane) {
        own(r0, lane & 3, x.f0);
        own(r1, lane & 3, x.f1);
        x.r0 = r0 + 4 * (lane & 3);
        x.r1 = r1 + 4 * (lane & 3);
    }
    __device__ static __forceinline__ void pair(Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c, th = c >> 1, gl = c & 1, sh = 4 - 2 * gl;
        if (gl == 0) {
            x.h0[0] = word_a2(x.r0 + 128 + 32 * th), x.h0[1] = word_a2(x.r0 + 144 + 32 * th);
            x.h1[0] = word_a2(x.r1 + 128 + 32 * th), x.h1[1] = word_a2(x.r1 + 144 + 32 * th);
        }
        const uint32_t CLO = dup16(0xE420u), CHI = dup16(0xD600u);   // -(1024 + 32), -(64 + 32)
        auto cv = [](uint32_t lo, uint32_t m1, uint32_t hi, uint32_t m2, uint32_t mg) { return and_or(lo, m1, and_or(hi, m2, mg)); };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t q0 = word_a2(x.r0 + 64 * th + 32 * gl + 16 * j), q1 = word_a2(x.r1 + 64 * th + 32 * gl + 16 * j);
            const uint32_t v0 = x.h0[j] << sh, v1 = x.h1[j] << sh, e0 = x.h0[j] >> (8 - sh), e1 = x.h1[j] >> (8 - sh);
            A[0][j][0] = hadd2(cv(q0, 0x000F000Fu, v0, 0x00300030u, 0x64006400u), CLO);
            A[0][j][1] = hadd2(cv(q1, 0x000F000Fu, v1, 0x00300030u, 0x64006400u), CLO);
            A[0][j][2] = hadd2(cv(q0 >> 8, 0x000F000Fu, e0, 0x00300030u, 0x64006400u), CLO);
            A[0][j][3] = hadd2(cv(q1 >> 8, 0x000F000Fu, e1, 0x00300030u, 0x64006400u), CLO);
            A[1][j][0] = hadd2(cv(q0, 0x00F000F0u, v0, 0x03000300u, 0x54005400u), CHI);
            A[1][j][1] = hadd2(cv(q1, 0x00F000F0u, v1, 0x03000300u, 0x54005400u), CHI);
            A[1][j][2] = hadd2(cv(q0 >> 8, 0x00F000F0u, e0, 0x03000300u, 0x54005400u), CHI);
            A[1][j][3] = hadd2(cv(q1 >> 8, 0x00F000F0u, e1, 0x03000300u, 0x54005400u), CHI);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s[b].f[0][h] = from(x.f0[2 * b + h], src);
                s[b].f[1][h] = from(x.f1[2 * b + h], src);
            }
    }
};

// The types of 32-weight blocks, BB bytes each: pair c is blocks 2c and 2c + 1.
template <int BB>
struct Blocks32 {
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        float d0[2], d1[2];   // the thread's own pair
        const uint8_t *r0, *r1;
    };
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane) {
        const int t = lane & 3;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            x.d0[b] = h2f(ld_u16(r0 + BB * (2 * t + b)));
            x.d1[b] = h2f(ld_u16(r1 + BB * (2 * t + b)));
        }
        x.r0 = r0;
        x.r1 = r1;
    }
    __device__ static __forceinline__ void scales(const Ctx& x, int src, Scale (&s)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            s[b].f[0][0] = from(x.d0[b], src);
            s[b].f[1][0] = from(x.d1[b], src);
        }
    }
};

template <> struct DU<T_Q8_0> : Blocks32<34> {
    static constexpr int UB = 8 * 34;
    static constexpr bool kW4 = false, kG16 = false, kMin = false;
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint32_t C = dup16(0xE480u);   // -(1024 + 128)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = 34 * (2 * c + b) + 2 + 8 * (lane & 3);
            const uint2 w0 = words2_a2(x.r0 + at), w1 = words2_a2(x.r1 + at);
            const uint32_t u0[2] = {w0.x, w0.y}, u1[2] = {w1.x, w1.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                A[b][j][0] = hadd2(and_xor(u0[j], 0x00FF00FFu, 0x64806480u), C);
                A[b][j][1] = hadd2(and_xor(u1[j], 0x00FF00FFu, 0x64806480u), C);
                A[b][j][2] = hadd2(and_xor(u0[j] >> 8, 0x00FF00FFu, 0x64806480u), C);
                A[b][j][3] = hadd2(and_xor(u1[j] >> 8, 0x00FF00FFu, 0x64806480u), C);
            }
        }
        scales(x, (lane & 28) | c, s);
    }
};

// Word t holds the low nibbles of weights 4t .. and the high ones of 16 + 4t ..
template <> struct DU<T_Q4_0> : Blocks32<18> {
    static constexpr int UB = 8 * 18;
    static constexpr bool kW4 = true, kG16 = false, kMin = false;
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint32_t LO = dup16(0xE408u), HI = dup16(0xD480u);   // -(1024 + 8), -(64 + 8)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = 18 * (2 * c + b) + 2 + 4 * (lane & 3);
            const uint32_t w0 = word_a2(x.r0 + at), w1 = word_a2(x.r1 + at);
            frag(A[b][0], w0, w1, 0x000F000Fu, 0x64006400u, LO, LO);
            frag(A[b][1], w0, w1, 0x00F000F0u, 0x54005400u, HI, HI);
        }
        scales(x, (lane & 28) | c, s);
    }
};

template <> struct DU<T_Q5_0> : Blocks32<22> {
    static constexpr int UB = 8 * 22;
    static constexpr bool kW4 = true, kG16 = false, kMin = false;
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint32_t C = dup16(0xE410u);   // -(1024 + 16)
        const int t = lane & 3;
        // code bytes: nibble | fifth bit << 4 (bit 4t + k of the word for byte k of step 0, 16 + 4t + k for step 1)
        auto lo = [&](uint32_t w, uint32_t q) { return and_or(w, 0x0F0F0F0Fu, HU<T_Q5_0>::spread(q >> (4 * t))); };
        auto hi = [&](uint32_t w, uint32_t q) { return and_or(w >> 4, 0x0F0F0F0Fu, HU<T_Q5_0>::spread(q >> (16 + 4 * t))); };
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = 22 * (2 * c + b) + 2;
            const uint32_t w0 = word_a2(x.r0 + at + 4 + 4 * t), w1 = word_a2(x.r1 + at + 4 + 4 * t);
            const uint32_t q0 = word_a2(x.r0 + at), q1 = word_a2(x.r1 + at);
            frag(A[b][0], lo(w0, q0), lo(w1, q1), 0x001F001Fu, 0x64006400u, C, C);
            frag(A[b][1], hi(w0, q0), hi(w1, q1), 0x001F001Fu, 0x64006400u, C, C);
        }
        scales(x, (lane & 28) | c, s);
    }
};

// Pair c: blocks 2c, 2c + 1 = half c / 2 of the super-block, code bits 2 j0 ..
// and 2 j0 + 2 .., j0 = 2 (c % 2); a block's halves are scaled on their own.
template <> struct DU<T_Q2_K> {
    static constexpr int UB = 84;
    static constexpr bool kW4 = true, kG16 = true, kMin = true;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        HU<T_Q2_K>::Row p0, p1;
        const uint8_t *r0, *r1;
    };
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane) {
        const int t = lane & 3;
        const float m0 = t & 1 ? 64.0f : 1024.0f, m1 = t & 1 ? 16.0f : 256.0f;
        x.p0 = HU<T_Q2_K>::row_params(r0, t, m0, m1);
        x.p1 = HU<T_Q2_K>::row_params(r1, t, m0, m1);
        x.r0 = r0 + 16 + 4 * t;
        x.r1 = r1 + 16 + 4 * t;
    }
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c;
        const bool up = c & 1;
        const uint32_t M[2] = {up ? 0x00300030u : 0x00030003u, up ? 0x00C000C0u : 0x000C000Cu};
        const uint32_t G[2] = {up ? 0x54005400u : 0x64006400u, up ? 0x4C004C00u : 0x5C005C00u};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w0 = lds32(x.r0 + 32 * (c >> 1) + 16 * j), w1 = lds32(x.r1 + 32 * (c >> 1) + 16 * j);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int k = 2 * b + j;
                frag(A[b][j], w0, w1, M[b], G[b], from(x.p0.cst[k], src), from(x.p1.cst[k], src));
                s[b].f[0][j] = from(x.p0.ds[k], src);
                s[b].f[1][j] = from(x.p1.ds[k], src);
                s[b].n[0][j] = -from(x.p0.r[k], src);
                s[b].n[1][j] = -from(x.p1.r[k], src);
            }
        }
    }
};

template <> struct DU<T_Q3_K> {
    static constexpr int UB = 110;
    static constexpr bool kW4 = true, kG16 = true, kMin = false;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        float f0[4], f1[4];
        uint32_t m0[2], m1[2];   // mask bits of the thread's words, all blocks
        const uint8_t *r0, *r1;
    };
    __device__ static __forceinline__ void own(const uint8_t* r, int t, float (&f)[4]) {
        const uint32_t l = word_a2(r + 96 + 4 * (t & 1)), u = word_a2(r + 104);
        const uint32_t S = ((l >> (4 * (t >> 1))) & 0x0F0F0F0Fu) | (((u >> (2 * t)) & 0x03030303u) << 4);
        const float d = h2f(ld_u16(r + 108));
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = d * (ubyte_f(S, k) - 32.0f);   // exact
    }
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane) {
        const int t = lane & 3;
        own(r0, t, x.f0);
        own(r1, t, x.f1);
        x.m0[0] = word_a2(r0 + 4 * t), x.m0[1] = word_a2(r0 + 16 + 4 * t);
        x.m1[0] = word_a2(r1 + 4 * t), x.m1[1] = word_a2(r1 + 16 + 4 * t);
        x.r0 = r0 + 32 + 4 * t;
        x.r1 = r1 + 32 + 4 * t;
    }
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c, tp = c >> 1, j0 = 2 * (c & 1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w0 = word_a2(x.r0 + 32 * tp + 16 * j), w1 = word_a2(x.r1 + 32 * tp + 16 * j);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // the code's two bits 2 jb .. of a byte, its mask bit moved from 4 tp + jb to 2 jb + 2; magic 2^(10 - 2 jb)
                const int jb = j0 + b;
                const uint32_t M = 0x00030003u << (2 * jb), B = 0x00040004u << (2 * jb);
                const uint32_t G = dup16(jb == 0 ? 0x6400u : jb == 1 ? 0x5C00u : jb == 2 ? 0x5400u : 0x4C00u);
                const uint32_t C = dup16(jb == 0 ? 0xE404u : jb == 1 ? 0xDC10u : jb == 2 ? 0xD440u : 0xCD00u);   // -(magic + 4)
                const int sh = 2 * jb + 2 - (4 * tp + jb);
                auto cv = [&](uint32_t w, uint32_t m) { return hadd2(and_or(w, M, and_or(HU<T_Q3_K>::shl(m, sh), B, G)), C); };
                A[b][j][0] = cv(w0, x.m0[j]);
                A[b][j][1] = cv(w1, x.m1[j]);
                A[b][j][2] = cv(w0 >> 8, x.m0[j] >> 8);
                A[b][j][3] = cv(w1 >> 8, x.m1[j] >> 8);
                s[b].f[0][j] = from(x.f0[2 * b + j], src);
                s[b].f[1][j] = from(x.f1[2 * b + j], src);
            }
        }
    }
};

// One unit of two tiles of rows (a0, a1 and b0, b1: rows g and g + 8 of each)
// against the same rows of x: y[0], y[1] += rows g, g + 8 against row t of x
// (NT = 4); y[0], y[1] row 2t and y[2], y[3] row 2t + 1 (NT = 8).  nvb: 32-blocks
// of the unit that exist.
template <int T, int NT>
__device__ __forceinline__ void run_unit(const uint8_t* a0, const uint8_t* a1, const uint8_t* b0, const uint8_t* b1,
                                         const uint8_t* xb, const float4* xm, int lane, int nvb, float (&ya)[NT / 2],
                                         float (&yb)[NT / 2]) {
    using D = DU<T>;
    const int g = lane >> 2, t = lane & 3;
    typename D::Ctx cx[2];
    D::load(cx[0], a0, a1, lane);
    D::load(cx[1], b0, b1, lane);
    const uint8_t* bp = NT == 4 ? xb + x_off<4>(0, g >> 1, g & 1) + 16 * t : xb + x_off<8>(0, g, 0) + 16 * t;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 B[2], L[2];
        float4 m[2][NT / 4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int blk = D::block(c, b);
            B[b] = lds128(bp + blk * (NT == 4 ? 512 : 1024));
            if (NT == 8) L[b] = lds128(bp + blk * 1024 + 512);
#pragma unroll
            for (int k = 0; k < NT / 4; ++k) m[b][k] = xm[blk * NT + (NT == 4 ? t : 2 * t + k)];
        }
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
            uint32_t A[2][2][4];
            Scale s[2];
            D::pair(cx[tile], c, lane, A, s);
            float(&y)[NT / 2] = tile ? yb : ya;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // a short last unit holds stale bytes behind its blocks
                if ((T == T_Q8_0 || T == T_Q5_0 || T == T_Q4_0) && D::block(c, b) >= nvb) continue;
                float C[2][4];
                mma16816_z(C[0], A[b][0][0], A[b][0][1], A[b][0][2], A[b][0][3], B[b].x, B[b].y);
                if constexpr (D::kG16) mma16816_z(C[1], A[b][1][0], A[b][1][1], A[b][1][2], A[b][1][3], B[b].z, B[b].w);
                else mma16816(C[0], A[b][1][0], A[b][1][1], A[b][1][2], A[b][1][3], B[b].z, B[b].w);
                if constexpr (NT == 8) {
                    mma16816(C[0], A[b][0][0], A[b][0][1], A[b][0][2], A[b][0][3], L[b].x, L[b].y);
                    mma16816(C[D::kG16], A[b][1][0], A[b][1][1], A[b][1][2], A[b][1][3], L[b].z, L[b].w);
                }
#pragma unroll
                for (int k = 0; k < NT / 4; ++k)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float& v = y[2 * k + r];
                        // this row of x: columns (hi, lo) of NT = 4, one column of NT = 8
                        auto sum = [&](int h) { return NT == 4 ? C[h][2 * r] + C[h][2 * r + 1] : C[h][2 * r + k]; };
                        const float4 x = m[b][k];
                        if constexpr (D::kG16) v = fmaf(x.y, fmaf(s[b].f[r][0], sum(0), s[b].f[r][1] * sum(1)), v);
                        else v = fmaf(s[b].f[r][0] * x.y, sum(0), v);
                        if constexpr (D::kMin) {
                            if constexpr (D::kG16) v = fmaf(s[b].n[r][0], x.z, fmaf(s[b].n[r][1], x.w, v));
                            else v = fmaf(s[b].n[r][0], x.x, v);
                        }
                    }
            }
        }
    }
}

}  // namespace dm
}  // namespace qk
