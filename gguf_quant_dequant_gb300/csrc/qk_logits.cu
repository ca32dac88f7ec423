// qk_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits, one pass over them.
//
//   y = x > 0 ? x / rep : x rep;  y -= freq c;  y -= pres     where the token
//   stands c > 0 times in the request's history and the row's drafted
//   ancestors;  y += bias;  -inf where the grammar bit is 0.
//
// The bound is the bytes: each logit read once and written once.  What may
// change a logit is sparse in the vocabulary, so a CTA takes one slice of
// some tokens and a group of consecutive rows and keeps one 32-bit word
// per token of the slice in shared memory: the count in the low 20 bits, 1 +
// the index of the token's (last) bias entry in the high 12.  The words are
// filled from the request's lists once and reused by its rows; a row's
// ancestors are added before its pass and taken out after it.  Integer
// atomics only, so the result does not depend on their order.
// 384 rows of 128,256 fp32 logits with grammar masks (401 MB): 89 us, 4.5 TB/s,
// 66 % of the measured copy rate; one row of 32,000: 5.0 us.  On
// top of the bytes a CTA reads its request's history before its first row,
// meets two barriers between rows, and, held to 32 registers by eight CTAs an SM,
// spills 84 bytes of stores and 108 of loads a thread in the vector path; their
// shares were not taken apart.  In that call a warp waits for loads (16.8 cycles an
// issue, spills among them) more than at barriers (4.2); DRAM is at 52 %.
#include <algorithm>
#include <cuda_bf16.h>

#include "qk_internal.h"
#include "qk_ptx.cuh"

namespace qk {
namespace lg {

constexpr int kThreads = 256, kPerSm = 8;   // CTAs on an SM
constexpr int kSliceMin = 512, kSliceMax = 6144;   // 8 x 24 KB of words fit an SM
constexpr int kCountBits = 20;
constexpr uint32_t kCountMask = (1u << kCountBits) - 1;

struct Args {
    const void* logits;
    int64_t n_rows, vocab, row_stride;
    const int32_t* cu;
    int n_req;
    const int32_t* hist;
    int64_t hist_stride;
    const int32_t* hist_len;
    const float *rep, *pres, *freq;
    const int32_t* draft;
    const uint64_t* mask;
    const int32_t* bias_tok;
    const float* bias_val;
    int64_t bias_stride;
    const int32_t* bias_len;
    const uint32_t* grammar;
    int64_t grammar_stride;
    void* out;
    int64_t out_stride;
    unsigned* status;
    int rows_per_cta, slice;
};

// First row of request r, inside [0, n_rows].
__device__ __forceinline__ int64_t row0_of(const Args& a, int r) {
    return min(max((int64_t)a.cu[r], (int64_t)0), a.n_rows);
}

template <bool BF16> struct Elem {
    using type = float;
    static constexpr int N = 4;   // elements of a 16-byte vector
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <> struct Elem<true> {
    using type = __nv_bfloat16;
    static constexpr int N = 8;
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// LONG: calls without masks whose chains could be longer than the words can
// count (a carry would reach the bias index).  A request that is has its drafts
// left out and is reported.  A variant of its own, because the look at it costs
// registers: in the ordinary kernel it took 384 x 128,256 logits from 89 to 108 us.
template <bool BF16, bool VEC, bool LONG>
__global__ void __launch_bounds__(kThreads, kPerSm) logits_kernel(const Args a) {
    using E = Elem<BF16>;
    using T = typename E::type;
    extern __shared__ __align__(16) uint32_t word[];
    const int tid = threadIdx.x;
    const int64_t v0 = (int64_t)blockIdx.x * a.slice;
    const int nv = (int)min((int64_t)a.slice, a.vocab - v0);
    const int64_t row_a = (int64_t)blockIdx.y * a.rows_per_cta, row_b = min(row_a + a.rows_per_cta, a.n_rows);
    int r = -1;
    int64_t r_lo = 0, r_hi = 0;   // rows the words stand for; none yet
    bool listed = false, drafted = false;   // a request's rows (else: rows of no request); with drafted tokens
    // A row's drafted ancestors that fall into the slice.
    auto ancestors = [&](int64_t row, uint32_t by) {
        const int64_t n = a.mask ? min((int64_t)64, r_hi - r_lo) : row - r_lo + 1;
        const uint64_t bits = a.mask ? a.mask[row] : 0;
        for (int64_t j = tid; j < n; j += kThreads)
            if (!a.mask || ((bits >> j) & 1)) {
                const int64_t t = a.draft[r_lo + j] - v0;
                if (t >= 0 && t < nv) atomicAdd(&word[t], by);
            }
    };
    float rep = 1.0f, pres = 0.0f, freq = 0.0f;
    for (int64_t row = row_a; row < row_b; ++row) {
        if (row >= r_hi) {   // another request: its lists
            // the last request that starts at or before the row
            int lo = -1, hi = a.n_req - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (row0_of(a, mid) <= row) lo = mid;
                else hi = mid - 1;
            }
            r = lo;
            listed = r >= 0 && row < row0_of(a, r + 1);
            r_lo = listed ? row0_of(a, r) : row;
            r_hi = listed ? row0_of(a, r + 1) : row + 1;
            drafted = listed && a.draft != nullptr;
            __syncthreads();
            for (int i = tid; i < a.slice; i += kThreads) word[i] = 0;
            __syncthreads();
            if (listed) {
                rep = a.rep[r];
                pres = a.pres[r];
                freq = a.freq[r];
                if (a.bias_tok) {
                    const int nb = (int)min((int64_t)a.bias_len[r], a.bias_stride);
                    const int32_t* bt = a.bias_tok + r * a.bias_stride;
                    for (int i = tid; i < nb; i += kThreads) {
                        const int64_t t = bt[i] - v0;
                        if (t >= 0 && t < nv) atomicMax(&word[t], (uint32_t)(i + 1) << kCountBits);
                    }
                    __syncthreads();
                }
                const int nh = (int)min((int64_t)a.hist_len[r], a.hist_stride);
                if constexpr (LONG) {
                    if (max(nh, 0) + (r_hi - r_lo) > (int64_t)kCountMask) {
                        drafted = false;
                        if (tid == 0) atomicOr(a.status, STATUS_BAD_COUNT);
                    }
                }
                const int32_t* ht = a.hist + r * a.hist_stride;
                for (int i = tid; i < nh; i += kThreads) {
                    const int64_t t = ht[i] - v0;
                    if (t >= 0 && t < nv) atomicAdd(&word[t], 1u);
                }
                if (drafted) ancestors(row, 1u);
            }
            __syncthreads();
        }
        const T* x = static_cast<const T*>(a.logits) + row * a.row_stride + v0;
        T* y = static_cast<T*>(a.out) + row * a.out_stride + v0;
        const uint32_t* gr = a.grammar ? a.grammar + row * a.grammar_stride + (v0 >> 5) : nullptr;
        auto one = [&](float v, uint32_t w, uint32_t allowed) {
            if (w) {
                const uint32_t c = w & kCountMask;
                if (c) {
                    v = v > 0.0f ? __fdiv_rn(v, rep) : v * rep;
                    v = __fsub_rn(__fsub_rn(v, __fmul_rn(freq, (float)c)), pres);
                }
                const uint32_t b = w >> kCountBits;
                if (b) v += a.bias_val[r * a.bias_stride + b - 1];
            }
            return allowed ? v : -INFINITY;
        };
        if constexpr (VEC) {
            constexpr int N = E::N;
            const int nvec = nv / N;
            // Two vectors at a time: with eight CTAs on an SM 64 KB of loads are in flight.
            for (int i0 = tid; i0 < nvec; i0 += 2 * kThreads) {
                uint4 u[2];
                const bool two = i0 + kThreads < nvec;
                u[0] = __ldcs(reinterpret_cast<const uint4*>(x) + i0);
                if (two) u[1] = __ldcs(reinterpret_cast<const uint4*>(x) + i0 + kThreads);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (k && !two) break;
                    const int i = i0 + k * kThreads;
                    const T* xe = reinterpret_cast<const T*>(&u[k]);
                    const uint32_t ok = gr ? gr[(i * N) >> 5] >> ((i * N) & 31) : ~0u;
                    uint4 o;
                    T* oe = reinterpret_cast<T*>(&o);
#pragma unroll
                    for (int j = 0; j < N; j += 4) {
                        const uint4 w = *reinterpret_cast<const uint4*>(&word[i * N + j]);
                        oe[j] = E::put(one(E::get(xe[j]), w.x, (ok >> j) & 1));
                        oe[j + 1] = E::put(one(E::get(xe[j + 1]), w.y, (ok >> (j + 1)) & 1));
                        oe[j + 2] = E::put(one(E::get(xe[j + 2]), w.z, (ok >> (j + 2)) & 1));
                        oe[j + 3] = E::put(one(E::get(xe[j + 3]), w.w, (ok >> (j + 3)) & 1));
                    }
                    __stcs(&reinterpret_cast<uint4*>(y)[i], o);
                }
            }
            for (int i = nvec * N + tid; i < nv; i += kThreads)
                y[i] = E::put(one(E::get(x[i]), word[i], gr ? (gr[i >> 5] >> (i & 31)) & 1 : 1u));
        } else {
#pragma unroll 2
            for (int i = tid; i < nv; i += kThreads)
                y[i] = E::put(one(E::get(x[i]), word[i], gr ? (gr[i >> 5] >> (i & 31)) & 1 : 1u));
        }
        if (drafted && row + 1 < min(row_b, r_hi)) {   // the words serve the next row
            __syncthreads();
            ancestors(row, 0u - 1u);
            ancestors(row + 1, 1u);
            __syncthreads();
        }
    }
}

template <bool BF16>
static cudaError_t launch_s(const Args& a, bool vec, cudaStream_t s) {
    const dim3 grid((unsigned)((a.vocab + a.slice - 1) / a.slice), (unsigned)((a.n_rows + a.rows_per_cta - 1) / a.rows_per_cta));
    const size_t smem = (size_t)a.slice * sizeof(uint32_t);
    if (a.draft && !a.mask && a.hist_stride + a.n_rows > (int64_t)kCountMask)
        logits_kernel<BF16, false, true><<<grid, kThreads, smem, s>>>(a);
    else if (vec) logits_kernel<BF16, true, false><<<grid, kThreads, smem, s>>>(a);
    else logits_kernel<BF16, false, false><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace lg

cudaError_t launch_logits_process(const LogitsArgs& p, int sms, cudaStream_t s) {
    lg::Args a{p.logits, p.n_rows, p.vocab, p.row_stride, p.cu, (int)p.n_req, p.hist, p.hist_stride, p.hist_len, p.rep,
               p.pres, p.freq, p.draft, p.mask, p.bias_tok, p.bias_val, p.bias_stride, p.bias_len, p.grammar,
               p.grammar_stride, p.out, p.out_stride, p.status, 1};
    // Rows of one request share the slice's words: as many rows per CTA as a
    // request has on average, at most 8, and at least what the grid's 65,535
    // row groups ask for.
    a.rows_per_cta = (int)std::max<int64_t>(std::min<int64_t>(8, std::max<int64_t>(1, p.n_rows / std::max<int64_t>(p.n_req, 1))),
                                            (p.n_rows + 65534) / 65535);
    // The slice: as long as one round of the GPU's CTAs allows (a CTA reads its
    // request's whole history), at most kSliceMax, then two rounds, three ...
    // 384 x 128,256 logits took 103 us in 1.26 rounds of 4,096-token slices.
    const int64_t groups = (p.n_rows + a.rows_per_cta - 1) / a.rows_per_cta, round = (int64_t)sms * lg::kPerSm;
    int64_t slice = lg::kSliceMax;
    for (int64_t w = 1; w <= 64; ++w) {
        const int64_t n = std::max<int64_t>(1, w * round / groups);
        slice = ((p.vocab + n - 1) / n + 31) / 32 * 32;   // whole words of the grammar mask
        if (slice <= lg::kSliceMax) break;
    }
    a.slice = (int)std::min<int64_t>(std::max<int64_t>(slice, lg::kSliceMin), lg::kSliceMax);
    const int es = p.bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
                     p.row_stride * es % 16 == 0 && p.out_stride * es % 16 == 0;
    return p.bf16 ? lg::launch_s<true>(a, vec, s) : lg::launch_s<false>(a, vec, s);
}

}  // namespace qk
