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
// Angles: pos * freq is kept as a whole number of 2^-96 turns, so that a far
// position loses nothing (fp32 would be a radian off near position 2^24); the
// cosine and sine come from their power series on an eighth of a turn, in
// pairs of fp32 (about 2^-40), and are rounded to fp32 once.  They are
// computed once per token and CTA and shared by its heads.
#include <algorithm>

#include "qk_internal.h"
#include "qk_paged.cuh"
#include "qk_ptx.cuh"
#include "qk_rows.cuh"

namespace qk {
namespace rope {

constexpr int kThreads = 256;
constexpr int kTable = 1024;   // (cos, sin) pairs a CTA can hold

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
    bool pairs, q_vec, k_vec, v_vec, qo_vec, ko_vec;
    void *q_out, *k_out;
    int64_t qo_stride, ko_stride;
    // the cache (keys and values go there when there is one)
    const int64_t* slots;
    uint8_t *K, *V;
    Pool pool;
    unsigned* status;
    int tok_per_cta, heads_per_cta;
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, bool vec, const float (&x)[8]) {
    if constexpr (BF16) {
        uint16_t* p = static_cast<uint16_t*>(base) + at;
        const uint4 w = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
        if (vec) {
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
        if (vec) {
            *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[i];
        }
    }
}

// T: the cache's block type, or 0 where keys go to rows.
template <int T, bool IN16, bool OUT16>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Args a) {
    __shared__ float2 table[kTable];
    const int tid = threadIdx.x, lanes = 1 << a.lanes_log2, sub = tid & (lanes - 1);
    const int heads = a.n_heads + a.n_kv + a.n_v, half = a.rot >> 1;
    const int64_t t0 = (int64_t)blockIdx.x * a.tok_per_cta;
    const int h0 = blockIdx.y * a.heads_per_cta;
    const int n_heads_here = min(a.heads_per_cta, heads - h0);
    const int n_tok_here = (int)min((int64_t)a.tok_per_cta, a.n_tok - t0);
    const int rows = n_tok_here * n_heads_here;
    for (int i = tid; i < n_tok_here * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        table[i] = cos_sin(turns_of(a.freq[f]), a.pos[t0 + t]);
    }
    __syncthreads();
    const int e0 = 8 * sub;                   // my elements of a row
    const int step = kThreads >> a.lanes_log2;
    const int rounds = (rows + step - 1) / step;
    for (int it = 0; it < rounds; ++it) {
        const int row = it * step + (tid >> a.lanes_log2);
        const bool live = row < rows;
        const int t = live ? row / n_heads_here : 0;
        const int head = live ? h0 + row - t * n_heads_here : 0;
        const int64_t tok = t0 + t;
        const int kind = !live ? 3 : head < a.n_heads ? 0 : head < a.n_heads + a.n_kv ? 1 : 2;   // query, key, value, none
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        const int g = head - (kind == 1 ? a.n_heads : kind == 2 ? a.n_heads + a.n_kv : 0);
        int64_t slot = -1;
        if (T != 0 && (kind == 1 || kind == 2)) {
            slot = a.slots[tok];
            if (slot < -1 || (slot >= 0 && (slot >> a.pool.page_log2) >= a.pool.n_pages)) {
                atomicOr(a.status, STATUS_BAD_PAGE);
                slot = -1;
            }
        }
        if (kind == 0) kv::load8<IN16>(a.q, tok * a.q_stride + (int64_t)g * a.d + e0, a.q_vec, x);
        if (kind == 1) kv::load8<IN16>(a.k, tok * a.k_stride + (int64_t)g * a.d + e0, a.k_vec, x);
        if (kind == 2) kv::load8<IN16>(a.v, tok * a.v_stride + (int64_t)g * a.d + e0, a.v_vec, x);
        const float* w = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
        if (__any_sync(0xffffffffu, w != nullptr)) {
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = __fmul_rn(x[i], x[i]);
            float sum = __fadd_rn(__fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])),
                                  __fadd_rn(__fadd_rn(s[4], s[5]), __fadd_rn(s[6], s[7])));
            for (int o = 1; o < lanes; o <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
            if (w) {
                const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)a.d), a.eps)));
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), w[e0 + i]);
            }
        }
        if (half > 0 && __any_sync(0xffffffffu, kind < 2)) {
            const bool turns = kind < 2 && e0 < a.rot;
            const float2* cs = table + t * half;
            if (a.pairs) {
                if (turns) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 r = cs[(e0 + i) >> 1];
                        const float u = x[i], v = x[i + 1];
                        x[i] = __fadd_rn(__fmul_rn(u, r.x), -__fmul_rn(v, r.y));
                        x[i + 1] = __fadd_rn(__fmul_rn(v, r.x), __fmul_rn(u, r.y));
                    }
                }
            } else {
                const bool second = e0 >= half;
                const int other = (tid & 31) + (turns ? (second ? -(half >> 3) : half >> 3) : 0);
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, x[i], other);
                if (turns) {
                    cs += second ? e0 - half : e0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 r = cs[i];
                        const float m = __fmul_rn(p[i], r.y);
                        x[i] = __fadd_rn(__fmul_rn(x[i], r.x), second ? m : -m);
                    }
                }
            }
        }
        if (kind == 0) store8<OUT16>(a.q_out, tok * a.qo_stride + (int64_t)g * a.d + e0, a.qo_vec, x);
        if constexpr (T == 0) {
            if (kind == 1) store8<OUT16>(a.k_out, tok * a.ko_stride + (int64_t)g * a.d + e0, a.ko_vec, x);
        } else if (__any_sync(0xffffffffu, kind == 1 || kind == 2)) {
            uint8_t* dst = nullptr;
            if (slot >= 0)
                dst = (kind == 1 ? a.K : a.V) + (sub >> 2) * Fmt<T>::BB +
                      pool_row(a.pool, slot >> a.pool.page_log2, g, (int)(slot & ((1 << a.pool.page_log2) - 1)));
            kv::append_block<T>(x, dst, sub & 3);
        }
    }
}

template <int T, bool IN16, bool OUT16>
static cudaError_t go(const Args& a, dim3 grid, cudaStream_t s) {
    rope_kernel<T, IN16, OUT16><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

static cudaError_t launch(int type, Args a, bool in16, bool out16, int sms, cudaStream_t s) {
    const int heads = a.n_heads + a.n_kv + a.n_v, lanes = a.d / 8;
    a.lanes_log2 = lanes == 4 ? 2 : lanes == 8 ? 3 : lanes == 16 ? 4 : 5;
    const int es = in16 ? 2 : 4, eo = out16 ? 2 : 4;
    auto vec = [](const void* p, int64_t stride, int e) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * e % 16 == 0; };
    a.q_vec = vec(a.q, a.q_stride, es);
    a.k_vec = vec(a.k, a.k_stride, es);
    a.v_vec = vec(a.v, a.v_stride, es);
    a.qo_vec = vec(a.q_out, a.qo_stride, eo);
    a.ko_vec = vec(a.k_out, a.ko_stride, eo);
    const int fit = kThreads / lanes;   // rows of one round
    if (heads < fit) {                  // several tokens a CTA
        a.tok_per_cta = std::min(fit / heads, kTable / std::max(a.rot / 2, 1));
        a.heads_per_cta = heads;
    } else {                            // a token a CTA, or for few tokens a round of its heads
        a.tok_per_cta = 1;
        a.heads_per_cta = a.n_tok >= 2 * sms ? heads : fit;
    }
    const dim3 grid((unsigned)((a.n_tok + a.tok_per_cta - 1) / a.tok_per_cta), (unsigned)((heads + a.heads_per_cta - 1) / a.heads_per_cta));
    switch (type) {
    case 0: return in16 ? (out16 ? go<0, true, true>(a, grid, s) : go<0, true, false>(a, grid, s))
                        : (out16 ? go<0, false, true>(a, grid, s) : go<0, false, false>(a, grid, s));
    case T_Q8_0: return in16 ? go<T_Q8_0, true, true>(a, grid, s) : go<T_Q8_0, false, true>(a, grid, s);
    case T_Q5_0: return in16 ? go<T_Q5_0, true, true>(a, grid, s) : go<T_Q5_0, false, true>(a, grid, s);
    case T_Q4_0: return in16 ? go<T_Q4_0, true, true>(a, grid, s) : go<T_Q4_0, false, true>(a, grid, s);
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
