// qk_rope.cu -- norms of query and key heads with the position rotation in
// the same pass: rows to rows (qk_norm_rope), or on the way into the paged
// cache (qk_kv_append_rope: keys and values quantized into their slots).
//
// A row of d elements belongs to d / 8 lanes, eight elements a lane.  Per row
//   inv = 1 / sqrt(sum x^2 / d + eps),  y = (x inv) w,
//   (a, b) -> (a cos - b sin, b cos + a sin)   for its rot / 2 pairs,
// every operation rounded to fp32 by itself (no fused multiply-add) and the
// sum of squares by neighbours (a lane's eight as a tree, then shuffles at
// distance 1, 2, 4 ..), so that a value, and the byte it is quantized to, does
// not depend on where or how it is computed.
//
// Angles: freq is kept as a whole number of 2^-96 turns, so that a far position
// loses nothing (fp32 would be a radian off near position 2^24); what is left of
// the angle, within an eighth of a turn, is held as two fp32 (2^-89 turns at
// worst, which only sines of angles below 2^-46 notice); the cosine and sine come
// from their power series there, in pairs of fp32 (about 2^-40), and are rounded
// to fp32 once.
//
// A warp takes a token and walks over its heads, 32 / (d / 8) rows a step, the
// next step's loads ahead of this one's arithmetic.  It computes the token's
// cosines and sines once (they cost some 200 instructions each) and keeps
// what its lanes need of them in registers for all heads; a CTA per token with
// the table in shared memory took 337 us for 32,764 tokens of 32 + 2 x 8 heads
// (d 128, Q4_0 pages), this takes 209.  The instructions bound it (about 150 a
// step with norm and rotation, 150 more where a step is quantized; the issue
// slots are 68 % used, DRAM 40 %): the bytes of that call would need 106 us.  Few tokens
// are bound by latency: 3.5 us for one token of 32 + 8 heads.
#include <algorithm>

#include "qk_internal.h"
#include "qk_paged.cuh"
#include "qk_ptx.cuh"
#include "qk_rows.cuh"

namespace qk {
namespace rope {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxHalf = 128;   // pairs of a row
constexpr int kCtas = 3;        // on an SM: 80 registers a thread (2: 32 % slower for 32,764 tokens, 5: 30 %, for what spills)
constexpr int kShares = 2;      // of the tokens' heads for each warp of the GPU (4: 20 % slower with 61 x 29 tokens)

// ---------------------------------------------------------------- angles --
// freq / (2 pi) as a fraction of a turn in units of 2^-96, modulo one turn
// (whole turns per position do not matter: positions are whole numbers):
// the 24-bit significand times the bits of 1 / (2 pi) that its exponent
// selects.  1 / (2 pi) to 192 bits.
struct Turn {
    uint64_t hi;   // units of 2^-64
    uint32_t lo;   // units of 2^-96
    bool ok;       // a finite frequency below 2^64
};
__device__ __forceinline__ Turn turns_of(float freq) {
    const uint32_t bits = __float_as_uint(freq);
    const int ex = (int)((bits >> 23) & 255u);
    const uint32_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int e = (ex ? ex : 1) - 150;   // freq = m 2^e
    Turn t{0, 0, ex != 255 && e <= 40};
    if (!t.ok) return t;
    // W = bits of 1 / (2 pi) from weight 2^(-e - 1) of the fraction down, 128 of them: floor(2^(128 + e) / (2 pi)) mod 2^128
    const uint64_t c[3] = {0x28BE60DB9391054Aull, 0x7F09D5F47D4D3770ull, 0x36D8A5664F10E410ull};
    const int sh = 64 - e;   // 192-bit value shifted right: 24 .. 213
    uint64_t w1 = 0, w0 = 0;   // high and low 64 bits of the low 128
    {
        const int q = sh >> 6, b = sh & 63;
        auto word = [&](int i) -> uint64_t { return i == 0 ? c[2] : i == 1 ? c[1] : i == 2 ? c[0] : 0ull; };   // from the lowest
        const uint64_t a0 = word(q), a1 = word(q + 1), a2 = word(q + 2);
        w0 = b ? (a0 >> b) | (a1 << (64 - b)) : a0;
        w1 = b ? (a1 >> b) | (a2 << (64 - b)) : a1;
    }
    // m W mod 2^128, then its top 96 bits
    const uint64_t p0 = w0 * m, p1 = w1 * m + __umul64hi(w0, m);
    t.hi = p1;
    t.lo = (uint32_t)(p0 >> 32);
    if (bits >> 31) {   // a negative frequency turns the other way
        t.lo = 0u - t.lo;
        t.hi = ~t.hi + (t.lo == 0u);
    }
    return t;
}

// Numbers as the sum of two fp32 (the second about 2^-24 of the first).
struct Two {
    float h, l;
};
__device__ __forceinline__ Two mul2(Two a, Two b) {
    const float p = __fmul_rn(a.h, b.h);
    return {p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h)};
}
// c + a b for |c| above |a b|.
__device__ __forceinline__ Two add_mul2(double c, Two a, Two b) {
    const float ch = (float)c, cl = (float)(c - (double)(float)c);   // constants: folded
    const Two p = mul2(a, b);
    const float s = __fadd_rn(ch, p.h);
    return {s, __fadd_rn(p.h, -__fadd_rn(s, -ch)) + (cl + p.l)};
}

// cos and sin of 2 pi pos freq, from the frequency in turns.
__device__ __forceinline__ float2 cos_sin(const Turn& t, int pos) {
    if (!t.ok) return make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
    // pos * turns, modulo one turn, for a signed pos
    const uint32_t n = (uint32_t)(pos < 0 ? -(int64_t)pos : pos);
    const uint64_t low = (uint64_t)t.lo * n;
    uint64_t hi = t.hi * n + (low >> 32);
    uint32_t lo = (uint32_t)low;
    if (pos < 0) {
        lo = 0u - lo;
        hi = ~hi + (lo == 0u);
    }
    // nearest quarter turn, and what is left: [-1/8, 1/8)
    const uint32_t quarter = (uint32_t)((hi + (1ull << 61)) >> 62) & 3u;
    const int64_t r = (int64_t)(hi - ((uint64_t)quarter << 62));
    const float rh = __ll2float_rn(r);
    const float rl = __ll2float_rn(r - __float2ll_rn(rh)) + (float)lo * 0x1p-32f;
    // y = 2 pi r 2^-64
    const Two x{rh * 0x1p-64f, rl * 0x1p-64f};
    constexpr double kTwoPi = 6.283185307179586476925;
    const float ph = (float)kTwoPi, pl = (float)(kTwoPi - (double)(float)kTwoPi);
    Two y = mul2(x, Two{ph, pl});
    {
        const float s = __fadd_rn(y.h, y.l);
        y.l = __fadd_rn(y.l, -__fadd_rn(s, -y.h));
        y.h = s;
    }
    const Two z = mul2(y, y);
    // sin y = y (1 - z/6 + z^2/120 - ..), cos y = 1 - z/2 + z^2/24 - ..; from z^4 on fp32 is enough (z <= 0.617)
    const float s4 = fmaf(z.h, fmaf(z.h, fmaf(z.h, -1.0f / 1307674368000.0f, 1.0f / 6227020800.0f), -1.0f / 39916800.0f), 1.0f / 362880.0f);
    const float c4 = fmaf(z.h, fmaf(z.h, fmaf(z.h, fmaf(z.h, 1.0f / 20922789888000.0f, -1.0f / 87178291200.0f), 1.0f / 479001600.0f),
                                    -1.0f / 3628800.0f), 1.0f / 40320.0f);
    const Two sn = mul2(y, add_mul2(1.0, z, add_mul2(-1.0 / 6, z, add_mul2(1.0 / 120, z, add_mul2(-1.0 / 5040, z, Two{s4, 0.0f})))));
    const Two cs = add_mul2(1.0, z, add_mul2(-0.5, z, add_mul2(1.0 / 24, z, add_mul2(-1.0 / 720, z, Two{c4, 0.0f}))));
    const float s = __fadd_rn(sn.h, sn.l), c = __fadd_rn(cs.h, cs.l);
    switch (quarter) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
    }
}

// ------------------------------------------------------------------ rows --
struct Args {
    const void *q, *k, *v;
    int64_t n_tok, q_stride, k_stride, v_stride;
    int n_heads, n_kv, n_v;   // rows of a token: queries, keys, values (n_v = 0 without a cache)
    int d, rot, lanes_log2;   // lanes of a row
    const int32_t* pos;
    const float *q_norm, *k_norm, *freq;
    float eps;
    bool pairs;
    void *q_out, *k_out;
    int64_t qo_stride, ko_stride;
    // the cache (keys and values go there when there is one)
    const int64_t* slots;
    uint8_t *K, *V;
    Pool pool;
    unsigned* status;
    int per;   // steps (32 / lanes rows each) of a warp per token
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
// Eight elements of a row as they lie in memory (VEC: 16-byte aligned).
template <bool BF16, bool VEC>
struct Raw {
    uint32_t w[BF16 ? 4 : 8];
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        if constexpr (BF16) {
            const uint16_t* p = static_cast<const uint16_t*>(base) + at;
            if (VEC) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
            }
        } else {
            const uint32_t* p = static_cast<const uint32_t*>(base) + at;
            if (VEC) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p)), v = __ldcs(reinterpret_cast<const uint4*>(p + 4));
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = p[i];
            }
        }
    }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = BF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u))
                        : make_float2(__uint_as_float(w[(2 * i) % (BF16 ? 4 : 8)]), __uint_as_float(w[(2 * i + 1) % (BF16 ? 4 : 8)]));
    }
};
template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&x)[8]) {
    if constexpr (BF16) {
        uint16_t* p = static_cast<uint16_t*>(base) + at;
        const uint4 w = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
        if (VEC) {
            *reinterpret_cast<uint4*>(p) = w;
        } else {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[2 * i] = (uint16_t)u[i];
                p[2 * i + 1] = (uint16_t)(u[i] >> 16);
            }
        }
    } else {
        float* p = static_cast<float*>(base) + at;
        if (VEC) {
            *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[i];
        }
    }
}

// Two products, and their sums with others, each rounded by itself. (The sums
// are not taken in pairs too: a paired product and a paired sum become one
// fused operation, whatever their roundings say.)
__device__ __forceinline__ float2 mul_rn(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add_rn(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

// T: the cache's block type, or 0 where keys go to rows.
template <int T, bool IN16, bool OUT16, bool VEC>
__global__ void __launch_bounds__(kThreads, kCtas) rope_kernel(const Args a) {
    __shared__ Turn turns[kMaxHalf];
    __shared__ float2 tables[kWarps][kMaxHalf];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lanes = 1 << a.lanes_log2, sub = lane & (lanes - 1), half = a.rot >> 1;
    const int rows = 32 >> a.lanes_log2;   // of a step
    const int e0 = 8 * sub;                // my elements of a row
    const int steps_q = (a.n_heads + rows - 1) / rows, steps_k = (a.n_kv + rows - 1) / rows, steps_v = (a.n_v + rows - 1) / rows;
    const int s0 = blockIdx.y * a.per, s1 = min(s0 + a.per, steps_q + steps_k + steps_v);
    for (int f = tid; f < half; f += kThreads) turns[f] = turns_of(a.freq[f]);
    __syncthreads();
    // The lane's rotation: y = x c + partner s.
    const bool turn = e0 < a.rot, second = e0 >= half;
    const int other = lane + (turn ? (second ? -(half >> 3) : half >> 3) : 0);
    float2* const table = tables[warp];
    const float inv_d = 1.0f / (float)a.d;   // d is a power of two: exact

    const int64_t tok = (int64_t)blockIdx.x * kWarps + warp;
    if (tok >= a.n_tok) return;
    const int pos = half > 0 ? a.pos[tok] : 0;
    int64_t slot = -1;
    if (T != 0 && s1 > steps_q) {
        slot = a.slots[tok];
        if (slot < -1 || (slot >= 0 && (slot >> a.pool.page_log2) >= a.pool.n_pages)) {
            if (lane == 0) atomicOr(a.status, STATUS_BAD_PAGE);
            slot = -1;
        }
    }
    // The token's cosines and sines, by the warp: y = x c + partner s.
    float2 c[4], sn[4];
    if (half > 0 && s0 < steps_q + steps_k) {
        for (int f = lane; f < half; f += 32) table[f] = cos_sin(turns[f], pos);
        __syncwarp();
        const float2* r = table + (a.pairs ? e0 >> 1 : second ? e0 - half : e0);
        if (turn) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 r0 = r[a.pairs ? i : 2 * i], r1 = r[a.pairs ? i : 2 * i + 1];
                c[i] = make_float2(r0.x, r1.x), sn[i] = make_float2(!a.pairs && second ? r0.y : -r0.y, a.pairs || second ? r1.y : -r1.y);
            }
        }
    }
    int first = 0;   // of the kind's steps
#pragma unroll 1
    for (int kind = 0; kind < (T == 0 ? 2 : 3); ++kind) {   // queries, keys, values
        const int n = kind == 0 ? a.n_heads : kind == 1 ? a.n_kv : a.n_v;
        const int last = first + (n + rows - 1) / rows;
        const int from = max(s0, first) - first, to = min(s1, last) - first;
        first = last;
        if (from >= to) continue;
        const float* norm = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
        float2 w[4];
        if (norm) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = make_float2(norm[e0 + 2 * i], norm[e0 + 2 * i + 1]);
        }
        const int g0 = from * rows + (lane >> a.lanes_log2);   // my head in the first step
        const int in_step = rows * a.d;
        const bool rows_out = kind == 0 || T == 0;
        int64_t in = tok * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + (int64_t)g0 * a.d + e0;
        const void* base = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        int64_t out = 0;   // elements, or bytes of the pool
        void* to_rows = kind == 0 ? a.q_out : a.k_out;
        uint8_t* pool = kind == 1 ? a.K : a.V;
        if (rows_out)
            out = tok * (kind == 0 ? a.qo_stride : a.ko_stride) + (int64_t)g0 * a.d + e0;
        else if constexpr (T != 0)
            out = (sub >> 2) * Fmt<T>::BB + pool_row(a.pool, slot >> a.pool.page_log2, g0, (int)(slot & ((1 << a.pool.page_log2) - 1)));
        const int64_t out_step = rows_out ? in_step : (int64_t)rows * a.pool.row_bytes << a.pool.page_log2;
        const bool turned = half > 0 && kind < 2;
        int left = n - g0;   // my head is one while this is above 0
        Raw<IN16, VEC> next{};
        if (left > 0) next.load(base, in);
#pragma unroll 1
        for (int st = from; st < to; ++st, left -= rows, out += out_step) {
            float2 x[4];
            next.get(x);
            in += in_step;
            if (st + 1 < to && left > rows) next.load(base, in);
            if (norm) {
                float2 q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = mul_rn(x[i], x[i]);
                float sum = __fadd_rn(__fadd_rn(__fadd_rn(q[0].x, q[0].y), __fadd_rn(q[1].x, q[1].y)),
                                      __fadd_rn(__fadd_rn(q[2].x, q[2].y), __fadd_rn(q[3].x, q[3].y)));
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 1));
                sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 2));
                if (lanes > 4) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 4));
                if (lanes > 8) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 8));
                if (lanes > 16) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, 16));
                const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, inv_d), a.eps)));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = mul_rn(mul_rn(x[i], make_float2(inv, inv)), w[i]);
            }
            if (turned) {
                float2 p[4];
                if (a.pairs) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = make_float2(x[i].y, x[i].x);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        p[i] = make_float2(__shfl_sync(0xffffffffu, x[i].x, other), __shfl_sync(0xffffffffu, x[i].y, other));
                }
                if (turn) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = add_rn(mul_rn(x[i], c[i]), mul_rn(p[i], sn[i]));
                }
            }
            const float y[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
            if (rows_out) {
                if (left > 0) store8<OUT16, VEC>(to_rows, out, y);
            } else if constexpr (T != 0) {
                kv::append_block<T>(y, left > 0 && slot >= 0 ? pool + out : nullptr, sub & 3);
            }
        }
    }
}

template <int T, bool IN16, bool OUT16>
static cudaError_t go(const Args& a, bool vec, dim3 grid, cudaStream_t s) {
    if (vec)
        rope_kernel<T, IN16, OUT16, true><<<grid, kThreads, 0, s>>>(a);
    else
        rope_kernel<T, IN16, OUT16, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

static cudaError_t launch(int type, Args a, bool in16, bool out16, int sms, cudaStream_t s) {
    const int lanes = a.d / 8;
    a.lanes_log2 = lanes == 4 ? 2 : lanes == 8 ? 3 : lanes == 16 ? 4 : 5;
    // 16-byte loads and stores, where all rows allow them.
    const int es = in16 ? 2 : 4, eo = out16 ? 2 : 4;
    auto fits = [](int n, const void* p, int64_t stride, int e) {
        return n == 0 || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * e % 16 == 0);
    };
    const bool vec = fits(a.n_heads, a.q, a.q_stride, es) && fits(a.n_kv, a.k, a.k_stride, es) && fits(a.n_v, a.v, a.v_stride, es) &&
                     fits(a.n_heads, a.q_out, a.qo_stride, eo) && (type != 0 || fits(a.n_kv, a.k_out, a.ko_stride, eo));
    // A warp takes a token's steps `per` at a time, so that there are about
    // kShares shares for each warp the GPU holds; each share computes the
    // token's cosines and sines again.
    const int rows = 32 / lanes;
    const int64_t steps = (a.n_heads + rows - 1) / rows + (a.n_kv + rows - 1) / rows + (a.n_v + rows - 1) / rows;
    const int64_t warps = (int64_t)sms * kCtas * kWarps;
    const int64_t per = std::min(steps, std::max<int64_t>(1, a.n_tok * steps / (kShares * warps)));
    const int64_t parts = (steps + per - 1) / per;
    a.per = (int)((steps + parts - 1) / parts);
    const dim3 grid((unsigned)((a.n_tok + kWarps - 1) / kWarps), (unsigned)((steps + a.per - 1) / a.per));
    switch (type) {
    case 0: return in16 ? (out16 ? go<0, true, true>(a, vec, grid, s) : go<0, true, false>(a, vec, grid, s))
                        : (out16 ? go<0, false, true>(a, vec, grid, s) : go<0, false, false>(a, vec, grid, s));
    case T_Q8_0: return in16 ? go<T_Q8_0, true, true>(a, vec, grid, s) : go<T_Q8_0, false, true>(a, vec, grid, s);
    case T_Q5_0: return in16 ? go<T_Q5_0, true, true>(a, vec, grid, s) : go<T_Q5_0, false, true>(a, vec, grid, s);
    case T_Q4_0: return in16 ? go<T_Q4_0, true, true>(a, vec, grid, s) : go<T_Q4_0, false, true>(a, vec, grid, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace rope

cudaError_t launch_norm_rope(const RopeArgs& r, void* k_out, bool out16, int64_t ko_stride, int sms, cudaStream_t s) {
    rope::Args a{};
    a.q = r.q, a.k = r.k, a.n_tok = r.n_tok, a.q_stride = r.q_stride, a.k_stride = r.k_stride;
    a.n_heads = r.n_heads, a.n_kv = r.n_kv, a.d = r.d, a.rot = r.rot, a.pos = r.pos;
    a.q_norm = r.q_norm, a.k_norm = r.k_norm, a.freq = r.freq, a.eps = r.eps, a.pairs = r.pairs;
    a.q_out = r.q_out, a.qo_stride = r.qo_stride, a.k_out = k_out, a.ko_stride = ko_stride;
    return rope::launch(0, a, r.bf16, out16, sms, s);
}

cudaError_t launch_kv_append_rope(int type, const RopeArgs& r, const void* v, int64_t v_stride, const int64_t* slots, uint8_t* K,
                                  uint8_t* V, int64_t n_pages, int page_log2, int row_bytes, unsigned* status, int sms,
                                  cudaStream_t s) {
    rope::Args a{};
    a.q = r.q, a.k = r.k, a.v = v, a.n_tok = r.n_tok, a.q_stride = r.q_stride, a.k_stride = r.k_stride, a.v_stride = v_stride;
    a.n_heads = r.n_heads, a.n_kv = r.n_kv, a.n_v = r.n_kv, a.d = r.d, a.rot = r.rot, a.pos = r.pos;
    a.q_norm = r.q_norm, a.k_norm = r.k_norm, a.freq = r.freq, a.eps = r.eps, a.pairs = r.pairs;
    a.q_out = r.q_out, a.qo_stride = r.qo_stride;
    a.slots = slots, a.K = K, a.V = V, a.pool = Pool{n_pages, page_log2, r.n_kv, row_bytes}, a.status = status;
    return rope::launch(type, a, r.bf16, true, sms, s);
}

}  // namespace qk
