// qk_tree.cu -- attention of drafted-token trees over the paged, block-
// quantized KV cache.
//
// For token i of request r, query head h and its kv head g:
//   s_t = scale q_h . K[t, g] over the visible t,  out = sum softmax(s)_t V[t, g].
// A CTA takes one request, one kv head and a range of kChunk positions; it
// decodes tiles of 32 positions to fp32 in shared memory and each warp keeps
// the running maximum, sum and value sum of four rows (token, head) at a
// time.  A second kernel joins the ranges (log-sum-exp, fixed order).
#include <algorithm>
#include <cuda_bf16.h>

#include "qk_formats.cuh"
#include "qk_internal.h"
#include "qk_paged.cuh"

namespace qk {
namespace tree {

constexpr int kWarps = 8, kTile = 32, kChunk = 2048, kRows = 4;

struct Args {
    const __nv_bfloat16* q;
    int64_t n_tok, q_stride;
    const uint8_t *K, *V;
    Pool pool;
    const int32_t* table;
    int64_t table_stride;
    const int32_t *ctx, *cu;
    const uint64_t* mask;
    int max_q, G, n_heads;
    float scale;
    __nv_bfloat16* out;
    int64_t out_stride;
    float* ws;          // [request][max_q][head][range][d + 2]
    int ranges;
    unsigned* status;
};

struct Req {
    int64_t tok0, ctx;
    int n;
};
__device__ __forceinline__ Req req_of(const Args& a, int r) {
    Req q;
    q.tok0 = min(max((int64_t)a.cu[r], (int64_t)0), a.n_tok);
    q.n = (int)min(max(min((int64_t)a.cu[r + 1], a.n_tok) - q.tok0, (int64_t)0), (int64_t)a.max_q);
    q.ctx = max(a.ctx[r], 0);
    return q;
}
__device__ __forceinline__ uint64_t seen_of(const Args& a, const Req& q, int i) {
    const uint64_t in = q.n >= 64 ? ~uint64_t(0) : (uint64_t(1) << q.n) - 1;
    return (a.mask ? a.mask[q.tok0 + i] : (i >= 63 ? ~uint64_t(0) : (uint64_t(2) << i) - 1)) & in;
}

template <int T, int D>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const Args a) {
    constexpr int NB = D / 32, E = D / 32, BB = Fmt<T>::BB;
    extern __shared__ float sm[];
    float* sk = sm;                       // [kTile][D + 1]
    float* sv = sm + kTile * (D + 1);     // [kTile][D]
    __shared__ int ids[kTile];
    const int r = blockIdx.z, g = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Req q = req_of(a, r);
    const int64_t total = q.ctx + q.n, p0 = (int64_t)blockIdx.x * kChunk, p1 = min(p0 + kChunk, total);
    const int rows = q.n * a.G;
    for (int rb = 0; rb < rows; rb += kWarps * kRows) {
        float m[kRows], l[kRows], acc[kRows][E], qv[kRows][E];
        uint64_t seen[kRows];
        for (int k = 0; k < kRows; ++k) {
            const int row = rb + warp * kRows + k;
            m[k] = -INFINITY;
            l[k] = 0.0f;
            seen[k] = row < rows ? seen_of(a, q, row / a.G) : 0;
            for (int e = 0; e < E; ++e) {
                acc[k][e] = 0.0f;
                qv[k][e] = row < rows ? __bfloat162float(a.q[(q.tok0 + row / a.G) * a.q_stride +
                                                             (g * a.G + row % a.G) * D + 32 * e + lane]) * a.scale : 0.0f;
            }
        }
        for (int64_t t0 = p0; t0 < p1; t0 += kTile) {
            const int nt = (int)min((int64_t)kTile, p1 - t0);
            __syncthreads();
            if (threadIdx.x < nt)
                ids[threadIdx.x] = page_of(a.pool, a.table + r * a.table_stride, a.table_stride, t0 + threadIdx.x, a.status);
            __syncthreads();
            for (int i = threadIdx.x; i < nt * NB * 2; i += kWarps * 32) {
                const int h = i & 1, b = (i >> 1) % NB, t = (i >> 1) / NB;
                if (ids[t] < 0) continue;
                const int off = (int)((t0 + t) & ((1 << a.pool.page_log2) - 1));
                const int64_t at = pool_row(a.pool, ids[t], g, off) + b * BB;
                float w[16];
                dequant_half<T>(a.K + at, 0, h, w);
                for (int j = 0; j < 16; ++j) sk[t * (D + 1) + 32 * b + 16 * h + j] = w[j];
                dequant_half<T>(a.V + at, 0, h, w);
                for (int j = 0; j < 16; ++j) sv[t * D + 32 * b + 16 * h + j] = w[j];
            }
            __syncthreads();
            for (int k = 0; k < kRows; ++k) {
                const int row = rb + warp * kRows + k;
                if (row >= rows) break;
                float s = 0.0f;
                for (int e = 0; e < E; ++e)
                    for (int c = 0; c < 32; ++c) s += __shfl_sync(0xffffffffu, qv[k][e], c) * (lane < nt ? sk[lane * (D + 1) + 32 * e + c] : 0.0f);
                const int64_t t = t0 + lane;
                const bool vis = lane < nt && ids[lane] >= 0 && (t < q.ctx || ((seen[k] >> (t - q.ctx)) & 1));
                s = vis ? s : -INFINITY;
                float mx = s;
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const unsigned any = __ballot_sync(0xffffffffu, vis);
                if (!any) continue;
                const float mn = fmaxf(m[k], mx), corr = m[k] == -INFINITY ? 0.0f : expf(m[k] - mn);
                const float p = vis ? expf(s - mn) : 0.0f;
                l[k] = l[k] * corr + p;   // this lane's share
                m[k] = mn;
                for (int e = 0; e < E; ++e) acc[k][e] *= corr;
                for (int c = 0; c < nt; ++c) {
                    if (!((any >> c) & 1)) continue;
                    const float pc = __shfl_sync(0xffffffffu, p, c);
                    for (int e = 0; e < E; ++e) acc[k][e] += pc * sv[c * D + 32 * e + lane];
                }
            }
        }
        if (p0 < p1)
            for (int k = 0; k < kRows; ++k) {
                const int row = rb + warp * kRows + k;
                if (row >= rows) break;
                float ls = l[k];
                for (int o = 16; o; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
                float* w = a.ws + ((((int64_t)r * a.max_q + row / a.G) * a.n_heads + g * a.G + row % a.G) * a.ranges + blockIdx.x) * (D + 2);
                for (int e = 0; e < E; ++e) w[32 * e + lane] = acc[k][e];
                if (lane == 0) {
                    w[D] = m[k];
                    w[D + 1] = ls;
                }
            }
    }
}

// One warp per (token, head): the ranges' sums on their common maximum.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
    constexpr int E = D / 32;
    const int64_t wid = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, r = blockIdx.y;
    const int i = (int)(wid / a.n_heads), h = (int)(wid % a.n_heads);
    const Req q = req_of(a, r);
    if (i >= q.n) return;
    const int ranges = (int)((q.ctx + q.n + kChunk - 1) / kChunk);
    const float* w = a.ws + (((int64_t)r * a.max_q + i) * a.n_heads + h) * a.ranges * (D + 2);
    float m = -INFINITY, l = 0.0f, acc[E] = {};
    for (int c = 0; c < ranges && c < a.ranges; ++c) m = fmaxf(m, w[c * (D + 2) + D]);
    for (int c = 0; c < ranges && c < a.ranges; ++c) {
        const float mc = w[c * (D + 2) + D];
        if (w[c * (D + 2) + D + 1] == 0.0f) continue;   // nothing visible in the range
        const float f = expf(mc - m);
        l += f * w[c * (D + 2) + D + 1];
        for (int e = 0; e < E; ++e) acc[e] += f * w[c * (D + 2) + 32 * e + lane];
    }
    __nv_bfloat16* o = a.out + (q.tok0 + i) * a.out_stride + h * D;
    for (int e = 0; e < E; ++e) o[32 * e + lane] = __float2bfloat16_rn(l == 0.0f ? 0.0f : acc[e] / l);
}

template <int T, int D>
static cudaError_t launch_t(const Args& a, int64_t n_req, cudaStream_t s) {
    const int smem = (kTile * (D + 1) + kTile * D) * (int)sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(tree_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    tree_kernel<T, D><<<dim3(a.ranges, a.pool.n_kv, (unsigned)n_req), kWarps * 32, smem, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    join_kernel<D><<<dim3((unsigned)((a.max_q * a.n_heads + 7) / 8), (unsigned)n_req), 256, 0, s>>>(a);
    return cudaGetLastError();
}
template <int T>
static cudaError_t launch_d(const Args& a, int64_t n_req, int d, cudaStream_t s) {
    switch (d) {
    case 32: return launch_t<T, 32>(a, n_req, s);
    case 64: return launch_t<T, 64>(a, n_req, s);
    case 128: return launch_t<T, 128>(a, n_req, s);
    case 256: return launch_t<T, 256>(a, n_req, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tree

int64_t attn_tree_ws_bytes(int64_t n_req, int max_q, int64_t max_pos, int n_heads, int d) {
    const int64_t ranges = std::max<int64_t>(1, (max_pos + tree::kChunk - 1) / tree::kChunk);
    return n_req * max_q * n_heads * ranges * (d + 2) * (int64_t)sizeof(float);
}

cudaError_t launch_attn_tree(int type, const void* q, int64_t n_tok, int64_t q_stride, const uint8_t* K, const uint8_t* V,
                             int64_t n_pages, int page_log2, int row_bytes, const int32_t* table, int64_t table_stride,
                             const int32_t* ctx, const int32_t* cu, const uint64_t* mask, int64_t n_req, int max_q,
                             int n_heads, int n_kv, int d, float scale, void* out, int64_t out_stride, void* ws,
                             unsigned* status, int sms, cudaStream_t s) {
    (void)sms;
    const int64_t ranges = std::max<int64_t>(1, ((table_stride << page_log2) + tree::kChunk - 1) / tree::kChunk);
    const tree::Args a{static_cast<const __nv_bfloat16*>(q), n_tok, q_stride, K, V, Pool{n_pages, page_log2, n_kv, row_bytes},
                       table, table_stride, ctx, cu, mask, max_q, n_heads / n_kv, n_heads, scale,
                       static_cast<__nv_bfloat16*>(out), out_stride, static_cast<float*>(ws), (int)ranges, status};
    switch (type) {
    case T_Q8_0: return tree::launch_d<T_Q8_0>(a, n_req, d, s);
    case T_Q5_0: return tree::launch_d<T_Q5_0>(a, n_req, d, s);
    case T_Q4_0: return tree::launch_d<T_Q4_0>(a, n_req, d, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace qk
