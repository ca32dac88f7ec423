// qk_dunits.cuh -- unit decoders for several activation rows at a time: 16
// weight rows x 256 weights against NT (4 or 8) rows of x, each weight
// converted once.
//
// Arithmetic: integer codes as exact fp16 A fragments, x as hi + lo fp16 terms
// after a power of two per 32-block, fp32 sums scaled per block.  Most types
// without a min hold the code less its offset (placed in the mantissa of a
// magic value and brought down by one exact add, as in qk_hunits.cuh).  The
// types with a min hold the code itself, as the fp16 subnormal whose bits it is:
// a shift and a mask and nothing else, the power of two goes into the scale; w =
// ds q - dm is then summed as ds sum(q x) - dm sum(x), so the error is a fraction
// of sum (|ds q| + |dm|) |x|.  (With the nearest code to dm / ds taken off first,
// as the decode GEMV does, it would be one of sum |w x|, for an add per two
// weights and its bookkeeping.)  Q6_K is summed that way too, dm = 32 ds: 8 %
// fewer instructions for its product, 4 % less time for a layer with it.
// The codes lie at bits 4 .. 7 (Q4_K), 3 .. 7, 2 .. 7 or 4 and 6 up, as high as
// costs little: an MMA adds products to a fixed number of places below the
// largest exponent, and a subnormal counts with the exponent that it is written
// with, so codes at the lowest bits lose what stands behind 2^-24 of 1 and not of
// themselves.  With Q4_K at bits 0 .. 3 and Q2_K at 0, 1, 4 and 5 a layer was 1.5e-6
// and 3e-6 of its norm off; now it is 2 to 5e-7, as with the other types, for 1 to
// 2 % more time.
// In qk_hunits.cuh a warp's four column groups hold four parts of K for one row
// of x; here all sixteen k of an MMA come from one 32-block and the eight
// columns are rows of x: four rows by (hi, lo), or eight rows with hi and lo in
// two MMAs.  So one MMA serves four rows instead of one, and a thread's sums are
// whole: row g and g + 8 against its own row(s) of x.
//
// Thread (g, t) supplies rows g and g + 8; of a 32-block's eight code words
// (four weights each) it takes words 2t and 2t + 1 in steps 0 and 1, or, where
// the weights are scaled by sixteens or the two halves sit in the nibbles of
// the same bytes (kW4), words t and t + 4, so that a step is one half of the
// block.  The scales of a pair of blocks are worked out by the thread whose
// group it was there (t = pair) and handed round the quad, by shuffles or, for
// Q4_K and Q5_K (kSc), through shared memory: two loads for eight shuffles, 7 %
// fewer instructions and 1 % less time.  (Q6_K's rings leave no room for it.)
#pragma once
#include <cstdint>

#include "qk_hunits.cuh"
#include "qk_hx.cuh"

namespace qk {
namespace dm {
using namespace hm;

// Prepared x of one unit: NT = 4 [block][row][plane][64 bytes], NT = 8
// [block][plane][row][64 bytes] (conflict-free for the B loads); the words of a
// plane in their order, or 0, 4, 1, 5, .. (kW4).  xm [block][row]: the block's
// sum twice (HALVES: its halves' sums, times -OFF 2^-22 where there is an offset),
// 2^e twice.
template <int NT>
__device__ __forceinline__ uint32_t x_off(int blk, int row, int plane) {
    return NT == 4 ? (uint32_t)(blk * 512 + row * 128 + plane * 64) : (uint32_t)(blk * 1024 + plane * 512 + row * 64);
}
constexpr int kXRow = 8 * 128;   // bytes of a row of x in a unit
template <int NT, bool W4, bool HALVES, int OFF>
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
    constexpr float kOff = OFF ? -(float)OFF * 0x1p-22f : 1.0f;
    if (q == 0) xm[blk * NT + row] = HALVES ? make_float4(kOff * m.z, kOff * m.w, m.y, m.y) : make_float4(m.x, m.x, m.y, m.y);
}

// Words of a row that starts on an even shared address: aligned words joined
// by a shift that is the row's own.
struct Even {
    const uint8_t* p;   // the word boundary at or before the row
    uint32_t sh;
    __device__ __forceinline__ void set(const uint8_t* r) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(r);
        p = reinterpret_cast<const uint8_t*>(a & ~uintptr_t(3));
        sh = (uint32_t)(a & 2) * 8;
    }
    // The word at byte o of the row (a multiple of 4), and the two from it on.
    __device__ __forceinline__ uint32_t word(int o) const { return __funnelshift_r(lds32(p + o), lds32(p + o + 4), sh); }
    __device__ __forceinline__ uint2 words(int o) const {
        const uint32_t w0 = lds32(p + o), w1 = lds32(p + o + 4), w2 = lds32(p + o + 8);
        return make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh));
    }
};
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

// Scales of a block as (row g, row g + 8): per half where scaled by sixteens
// (else [0] alone), and the negative mins of the types with a min.
struct Scale {
    float2 f[2], n[2];
};

// A decoder: UB bytes per row and unit, kW4 (above), kG16 (scaled by
// sixteens), kMin (has a min), kSc (scales through shared memory), kOff (codes less
// this; 0: the fragments have it off), block(pair c, b), Ctx, load(ctx, r0, r1, lane),
// pair(ctx, c, lane, A, s): fragments A[b][step] and scales s[b] of the pair's
// two blocks; pairs are taken in their order.
template <int T> struct DU;

// Q4_K and Q5_K: d * sc and dmin * m of the thread's own pair of blocks, the
// first by 2^BITS (the codes' place).
struct RowMin {
    float2 ds, ndm;
};
template <int BITS>
__device__ __forceinline__ RowMin row_min(const uint4& h, int t) {
    const uint32_t f = HU<T_Q4_K>::fields(h, t);
    const float d = h2f(h.x & 0xFFFFu), dmin = h2f(h.x >> 16);
    constexpr float kM = 8388608.0f;   // 2^23
    auto two = [&](uint32_t s0, uint32_t s1) {
        return __fadd2_rn(make_float2(__uint_as_float(__byte_perm(f, 0x4B000000u, s0)), __uint_as_float(__byte_perm(f, 0x4B000000u, s1))),
                          make_float2(-kM, -kM));
    };
    const float up = d * (float)(1 << BITS);
    return {__fmul2_rn(make_float2(up, up), two(0x7650, 0x7651)),
            __fmul2_rn(make_float2(-dmin, -dmin), two(0x7652, 0x7653))};
}
// The scales of a tile's rows in shared memory, [pair][g][2]: ds of both blocks
// and -dm of both, of rows g and g + 8 side by side as they are used.
constexpr int kScalePitch = 18;   // of a pair
__device__ __forceinline__ void put_scales(float4* sc, int lane, const RowMin& p0, const RowMin& p1) {
    sc += (lane & 3) * kScalePitch + 2 * (lane >> 2);
    sc[0] = make_float4(p0.ds.x, p1.ds.x, p0.ds.y, p1.ds.y);
    sc[1] = make_float4(p0.ndm.x, p1.ndm.x, p0.ndm.y, p1.ndm.y);
}
__device__ __forceinline__ void scales_min(const float4* sc, int c, Scale (&s)[2]) {
    const float4 u = sc[c * kScalePitch], v = sc[c * kScalePitch + 1];
    s[0].f[0] = make_float2(u.x, u.y);
    s[1].f[0] = make_float2(u.z, u.w);
    s[0].n[0] = make_float2(v.x, v.y);
    s[1].n[0] = make_float2(v.z, v.w);
}
// Four A registers each of the low and the high nibbles, at bits 4 .. 7.
__device__ __forceinline__ void nibbles(uint32_t (&lo)[4], uint32_t (&hi)[4], uint32_t w0, uint32_t w1) {
    constexpr uint32_t M = 0x00F000F0u;
    lo[0] = (w0 << 4) & M;
    lo[1] = (w1 << 4) & M;
    lo[2] = (w0 >> 4) & M;
    lo[3] = (w1 >> 4) & M;
    hi[0] = w0 & M;
    hi[1] = w1 & M;
    hi[2] = (w0 >> 8) & M;
    hi[3] = (w1 >> 8) & M;
}
// Four A registers of code bytes.
__device__ __forceinline__ void frag_bytes(uint32_t (&A)[4], uint32_t w0, uint32_t w1) {
    A[0] = __byte_perm(w0, 0u, 0x4240u);
    A[1] = __byte_perm(w1, 0u, 0x4240u);
    A[2] = __byte_perm(w0, 0u, 0x4341u);
    A[3] = __byte_perm(w1, 0u, 0x4341u);
}

template <> struct DU<T_Q4_K> {
    static constexpr int UB = 144, kOff = 0;
    static constexpr bool kW4 = false, kG16 = false, kMin = true, kSc = true;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        const float4* sc;
        const uint8_t *r0, *r1;
    };
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane, float4* sc) {
        put_scales(sc, lane, row_min<20>(lds128(r0), lane & 3), row_min<20>(lds128(r1), lane & 3));
        x.sc = sc + 2 * (lane >> 2);
        x.r0 = r0 + 16 + 8 * (lane & 3);
        x.r1 = r1 + 16 + 8 * (lane & 3);
    }
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint2 w0 = lds64(x.r0 + 32 * c), w1 = lds64(x.r1 + 32 * c);
        nibbles(A[0][0], A[1][0], w0.x, w1.x);
        nibbles(A[0][1], A[1][1], w0.y, w1.y);
        scales_min(x.sc, c, s);
    }
};

template <> struct DU<T_Q5_K> {
    static constexpr int UB = 176, kOff = 0;
    static constexpr bool kW4 = false, kG16 = false, kMin = true, kSc = true;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        const float4* sc;
        const uint8_t *r0, *r1;
        uint2 v0, v1;   // the fifth bits of the thread's words, four bits up, moved down two bits a pair
    };
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane, float4* sc) {
        put_scales(sc, lane, row_min<21>(lds128(r0), lane & 3), row_min<21>(lds128(r1), lane & 3));
        x.sc = sc + 2 * (lane >> 2);
        x.v0 = lds64(r0 + 16 + 8 * (lane & 3));
        x.v1 = lds64(r1 + 16 + 8 * (lane & 3));
        x.r0 = r0 + 48 + 8 * (lane & 3);
        x.r1 = r1 + 48 + 8 * (lane & 3);
    }
    // Code bytes, at bits 3 .. 7, of the low and high nibbles with their fifth bits (bits 0 and 1 of v's bytes).
    __device__ static __forceinline__ uint32_t low(uint32_t w, uint32_t v) { return and_or(w << 3, 0x78787878u, (v << 7) & 0x80808080u); }
    __device__ static __forceinline__ uint32_t high(uint32_t w, uint32_t v) { return and_or(w >> 1, 0x78787878u, (v << 6) & 0x80808080u); }
    __device__ static __forceinline__ void pair(Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint2 w0 = lds64(x.r0 + 32 * c), w1 = lds64(x.r1 + 32 * c);
        frag_bytes(A[0][0], low(w0.x, x.v0.x), low(w1.x, x.v1.x));
        frag_bytes(A[0][1], low(w0.y, x.v0.y), low(w1.y, x.v1.y));
        frag_bytes(A[1][0], high(w0.x, x.v0.x), high(w1.x, x.v1.x));
        frag_bytes(A[1][1], high(w0.y, x.v0.y), high(w1.y, x.v1.y));
        x.v0.x >>= 2, x.v0.y >>= 2, x.v1.x >>= 2, x.v1.y >>= 2;
        scales_min(x.sc, c, s);
    }
};

// Pair c: the 32-blocks (th, gl) and (th, gl + 2), th = c / 2, gl = c % 2, of
// low and high nibbles of the same bytes.  Codes 0 .. 63 as they are: their
// offset, 32, goes into the sums of x.
template <> struct DU<T_Q6_K> {
    static constexpr int UB = 210, kOff = 32;
    static constexpr bool kW4 = true, kG16 = true, kMin = false, kSc = false;
    __device__ static __forceinline__ int block(int c, int b) { return 4 * (c >> 1) + (c & 1) + 2 * b; }
    struct Ctx {
        float f0[4], f1[4];   // d * scale * 2^22 of the thread's own pair: block, half
        Even r0, r1;
        uint32_t h0[2], h1[2];   // high bits of the current half
    };
    __device__ static __forceinline__ void own(const uint8_t* r, int t, float (&f)[4]) {
        const int at = 8 * (t >> 1) + 2 * (t & 1);
        const uint32_t u = (ld_u16(r + 192 + at) | (ld_u16(r + 196 + at) << 16)) ^ 0x80808080u;   // + 128
        const float d = h2f(ld_u16(r + 208)) * 0x1p22f;
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = d * (ubyte_f(u, k) - 128.0f);   // exact
    }
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane, float4* sc) {
        own(r0, lane & 3, x.f0);
        own(r1, lane & 3, x.f1);
        x.r0.set(r0 + 4 * (lane & 3));
        x.r1.set(r1 + 4 * (lane & 3));
    }
    __device__ static __forceinline__ void pair(Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c, th = c >> 1, gl = c & 1, sh = 2 * gl;
        if (gl == 0) {
            x.h0[0] = x.r0.word(128 + 32 * th), x.h0[1] = x.r0.word(144 + 32 * th);
            x.h1[0] = x.r1.word(128 + 32 * th), x.h1[1] = x.r1.word(144 + 32 * th);
        }
        // four code bytes, at bits 2 .. 7: a nibble each, and two bits
        auto code = [](uint32_t low, uint32_t high) { return and_or(low, 0x3C3C3C3Cu, high & 0xC0C0C0C0u); };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t q0 = x.r0.word(64 * th + 32 * gl + 16 * j), q1 = x.r1.word(64 * th + 32 * gl + 16 * j);
            const uint32_t k0 = code(q0 << 2, x.h0[j] << (6 - sh)), k1 = code(q1 << 2, x.h1[j] << (6 - sh));
            const uint32_t n0 = code(q0 >> 2, x.h0[j] << (2 - sh)), n1 = code(q1 >> 2, x.h1[j] << (2 - sh));
            frag_bytes(A[0][j], k0, k1);
            frag_bytes(A[1][j], n0, n1);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s[b].f[h] = make_float2(from(x.f0[2 * b + h], src), from(x.f1[2 * b + h], src));
            }
    }
};

// The types of 32-weight blocks, BB bytes each: pair c is blocks 2c and 2c + 1.
template <int BB>
struct Blocks32 {
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        float d0[2], d1[2];   // the thread's own pair
        Even q0[2], q1[2];    // behind the scales of the first pair's blocks; a pair is a multiple of 4 bytes
    };
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane, float4* sc) {
        static_assert(2 * BB % 4 == 0, "pairs keep the alignment");
        const int t = lane & 3;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            x.d0[b] = h2f(ld_u16(r0 + BB * (2 * t + b)));
            x.d1[b] = h2f(ld_u16(r1 + BB * (2 * t + b)));
            x.q0[b].set(r0 + BB * b + 2);
            x.q1[b].set(r1 + BB * b + 2);
        }
    }
    __device__ static __forceinline__ void scales(const Ctx& x, int src, Scale (&s)[2]) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            s[b].f[0] = make_float2(from(x.d0[b], src), from(x.d1[b], src));
        }
    }
};

template <> struct DU<T_Q8_0> : Blocks32<34> {
    static constexpr int UB = 8 * 34, kOff = 0;
    static constexpr bool kW4 = false, kG16 = false, kMin = false, kSc = false;
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint32_t C = dup16(0xE480u);   // -(1024 + 128)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = 68 * c + 8 * (lane & 3);
            const uint2 w0 = x.q0[b].words(at), w1 = x.q1[b].words(at);
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
    static constexpr int UB = 8 * 18, kOff = 0;
    static constexpr bool kW4 = true, kG16 = false, kMin = false, kSc = false;
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint32_t LO = dup16(0xE408u), HI = dup16(0xD480u);   // -(1024 + 8), -(64 + 8)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = 36 * c + 4 * (lane & 3);
            const uint32_t w0 = x.q0[b].word(at), w1 = x.q1[b].word(at);
            frag(A[b][0], w0, w1, 0x000F000Fu, 0x64006400u, LO, LO);
            frag(A[b][1], w0, w1, 0x00F000F0u, 0x54005400u, HI, HI);
        }
        scales(x, (lane & 28) | c, s);
    }
};

template <> struct DU<T_Q5_0> : Blocks32<22> {
    static constexpr int UB = 8 * 22, kOff = 0;
    static constexpr bool kW4 = true, kG16 = false, kMin = false, kSc = false;
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const uint32_t C = dup16(0xE410u);   // -(1024 + 16)
        const int t = lane & 3;
        // code bytes: nibble | fifth bit << 4 (bit 4t + k of the word for byte k of step 0, 16 + 4t + k for step 1)
        auto lo = [&](uint32_t w, uint32_t q) { return and_or(w, 0x0F0F0F0Fu, HU<T_Q5_0>::spread(q >> (4 * t))); };
        auto hi = [&](uint32_t w, uint32_t q) { return and_or(w >> 4, 0x0F0F0F0Fu, HU<T_Q5_0>::spread(q >> (16 + 4 * t))); };
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t w0 = x.q0[b].word(44 * c + 4 + 4 * t), w1 = x.q1[b].word(44 * c + 4 + 4 * t);
            const uint32_t q0 = x.q0[b].word(44 * c), q1 = x.q1[b].word(44 * c);
            frag(A[b][0], lo(w0, q0), lo(w1, q1), 0x001F001Fu, 0x64006400u, C, C);
            frag(A[b][1], hi(w0, q0), hi(w1, q1), 0x001F001Fu, 0x64006400u, C, C);
        }
        scales(x, (lane & 28) | c, s);
    }
};

// Pair c: blocks 2c, 2c + 1 = half c / 2 of the super-block, code bits 2 j0 ..
// and 2 j0 + 2 .., j0 = 2 (c % 2); a block's halves are scaled on their own.
template <> struct DU<T_Q2_K> {
    static constexpr int UB = 84, kOff = 0;
    static constexpr bool kW4 = true, kG16 = true, kMin = true, kSc = false;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        float f0[4], f1[4], n0[4], n1[4];   // of the thread's own pair: block, half; scales by 2^20 and 2^18 (the codes' places)
        const uint8_t *r0, *r1;
    };
    __device__ static __forceinline__ void own(const uint8_t* r, int t, float (&f)[4], float (&n)[4]) {
        const uint32_t sm = lds32(r + 4 * t), dd = lds32(r + 80);   // (scale, min) bytes; d, dmin
        const uint32_t sc = sm & 0x0F0F0F0Fu, mn = (sm >> 4) & 0x0F0F0F0Fu;
        const float d = h2f(dd & 0xFFFFu) * 0x1p20f, dmin = h2f(dd >> 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = (k < 2 ? d : d * 0.25f) * ubyte_f(sc, k);
            n[k] = -dmin * ubyte_f(mn, k);
        }
    }
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane, float4* sc) {
        const int t = lane & 3;
        own(r0, t, x.f0, x.n0);
        own(r1, t, x.f1, x.n1);
        x.r0 = r0 + 16 + 4 * t;
        x.r1 = r1 + 16 + 4 * t;
    }
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c;
        const int sh = c & 1 ? 0 : 4;   // to bits 4 .. 7
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w0 = lds32(x.r0 + 32 * (c >> 1) + 16 * j), w1 = lds32(x.r1 + 32 * (c >> 1) + 16 * j);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int k = 2 * b + j;
                const uint32_t M = b ? 0x00C000C0u : 0x00300030u;
                A[b][j][0] = (w0 << sh) & M;
                A[b][j][1] = (w1 << sh) & M;
                A[b][j][2] = (w0 >> (8 - sh)) & M;
                A[b][j][3] = (w1 >> (8 - sh)) & M;
                s[b].f[j] = make_float2(from(x.f0[k], src), from(x.f1[k], src));
                s[b].n[j] = make_float2(from(x.n0[k], src), from(x.n1[k], src));
            }
        }
    }
};

template <> struct DU<T_Q3_K> {
    static constexpr int UB = 110, kOff = 0;
    static constexpr bool kW4 = true, kG16 = true, kMin = false, kSc = false;
    __device__ static __forceinline__ int block(int c, int b) { return 2 * c + b; }
    struct Ctx {
        float f0[4], f1[4];
        uint32_t m0[2], m1[2];   // mask bits of the thread's words, all blocks
        Even r0, r1;             // from byte 4t on
    };
    __device__ static __forceinline__ void own(const uint8_t* r, int t, float (&f)[4]) {
        Even w;
        w.set(r);
        const uint32_t l = w.word(96 + 4 * (t & 1)), u = w.word(104);
        const uint32_t S = ((l >> (4 * (t >> 1))) & 0x0F0F0F0Fu) | (((u >> (2 * t)) & 0x03030303u) << 4);
        const float d = h2f(ld_u16(r + 108));
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = d * (ubyte_f(S, k) - 32.0f);   // exact
    }
    __device__ static __forceinline__ void load(Ctx& x, const uint8_t* r0, const uint8_t* r1, int lane, float4* sc) {
        const int t = lane & 3;
        own(r0, t, x.f0);
        own(r1, t, x.f1);
        x.r0.set(r0 + 4 * t);
        x.r1.set(r1 + 4 * t);
        x.m0[0] = x.r0.word(0), x.m0[1] = x.r0.word(16);
        x.m1[0] = x.r1.word(0), x.m1[1] = x.r1.word(16);
    }
    __device__ static __forceinline__ void pair(const Ctx& x, int c, int lane, uint32_t (&A)[2][2][4], Scale (&s)[2]) {
        const int src = (lane & 28) | c, tp = c >> 1, j0 = 2 * (c & 1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w0 = x.r0.word(32 + 32 * tp + 16 * j), w1 = x.r1.word(32 + 32 * tp + 16 * j);
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
                s[b].f[j] = make_float2(from(x.f0[2 * b + j], src), from(x.f1[2 * b + j], src));
            }
        }
    }
};

// One unit of two tiles of rows (a0, a1 and b0, b1: rows g and g + 8 of each)
// against the same rows of x: y[0] += (row g, row g + 8) against row t of x (NT =
// 4); y[0] against row 2t and y[1] against row 2t + 1 (NT = 8).  nvb: 32-blocks of
// the unit that exist.
template <int T, int NT>
__device__ __forceinline__ void run_unit(const uint8_t* a0, const uint8_t* a1, const uint8_t* b0, const uint8_t* b1,
                                         const uint8_t* xb, const float4* xm, float4* sc, int lane, int nvb, float2 (&ya)[NT / 4],
                                         float2 (&yb)[NT / 4]) {
    using D = DU<T>;
    const int g = lane >> 2, t = lane & 3;
    typename D::Ctx cx[2];
    D::load(cx[0], a0, a1, lane, sc);
    D::load(cx[1], b0, b1, lane, sc + 4 * kScalePitch);
    if (D::kSc) __syncwarp();
    const uint8_t* bp = NT == 4 ? xb + x_off<4>(0, g >> 1, g & 1) + 16 * t : xb + x_off<8>(0, g, 0) + 16 * t;
    // Half of the pairs unrolled: the code of all four is fetched longer than it runs where few units follow one another.
#pragma unroll 1
    for (int c2 = 0; c2 < 4; c2 += 2) {
#pragma unroll
        for (int c1 = 0; c1 < 2; ++c1) {
            const int c = c2 + c1;
            uint4 B[2], L[2];
            float4 m[2][NT / 4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int blk = D::block(c, b);
                B[b] = lds128(bp + blk * (NT == 4 ? 512 : 1024));
                if (NT == 8) L[b] = lds128(bp + blk * 1024 + 512);
#pragma unroll
                for (int k = 0; k < NT / 4; ++k) {
                    const float4* p = xm + blk * NT + (NT == 4 ? t : 2 * t + k);
                    if constexpr (D::kMin || D::kOff) {
                        m[b][k] = *p;
                    } else {
                        const float2 up = reinterpret_cast<const float2*>(p)[1];
                        m[b][k] = make_float4(0.0f, 0.0f, up.x, up.y);
                    }
                }
            }
#pragma unroll
            for (int tile = 0; tile < 2; ++tile) {
                uint32_t A[2][2][4];
                Scale s[2];
                D::pair(cx[tile], c, lane, A, s);
                float2(&y)[NT / 4] = tile ? yb : ya;
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
                    for (int k = 0; k < NT / 4; ++k) {
                        // rows g, g + 8 against this row of x: columns (hi, lo) of NT = 4, one column of NT = 8
                        auto sum = [&](int h) {
                            return NT == 4 ? make_float2(C[h][0] + C[h][1], C[h][2] + C[h][3]) : make_float2(C[h][k], C[h][2 + k]);
                        };
                        const float4 x = m[b][k];
                        const float2 up = make_float2(x.z, x.w);
                        if constexpr (D::kOff)
                            y[k] = __ffma2_rn(s[b].f[0], __ffma2_rn(sum(0), up, make_float2(x.x, x.x)),
                                              __ffma2_rn(s[b].f[1], __ffma2_rn(sum(1), up, make_float2(x.y, x.y)), y[k]));
                        else if constexpr (D::kG16) y[k] = __ffma2_rn(up, __ffma2_rn(s[b].f[0], sum(0), __fmul2_rn(s[b].f[1], sum(1))), y[k]);
                        else y[k] = __ffma2_rn(s[b].f[0], __fmul2_rn(sum(0), up), y[k]);
                        if constexpr (D::kMin) {
                            if constexpr (D::kG16) {
                                y[k] = __ffma2_rn(s[b].n[0], make_float2(x.x, x.x), __ffma2_rn(s[b].n[1], make_float2(x.y, x.y), y[k]));
                            } else {
                                y[k] = __ffma2_rn(s[b].n[0], make_float2(x.x, x.y), y[k]);
                            }
                        }
                    }
                }
            }
        }
    }
}

}  // namespace dm
}  // namespace qk
