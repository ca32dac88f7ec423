// qk_moe.cu -- a mixture-of-experts layer (qk_moe_ffn): the router, the last
// sum, and the launches of the layer.
#include <cooperative_groups.h>

#include "qk_internal.h"
#include "qk_moe.cuh"

namespace cg = cooperative_groups;

namespace qk {
namespace moe {

// Order-preserving image of a float: one for both zeros, NaN above all.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v), mag = u & 0x7fffffffu;
    if (mag > 0x7f800000u) return 0xffffffffu;
    return (u >> 31) && mag ? ~u : mag | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// One warp, one token: the k largest of n logits (logit(e); the lowest index of
// equals), their softmax over all n or over the k.
template <int NE, class F>
__device__ __forceinline__ void choose(F logit, int n, int k, bool norm, float scale, int lane, int32_t* ids, float* gate) {
    uint32_t key[NE];
    float l[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < n ? logit(e) : -INFINITY;
        key[i] = e < n ? key_of(l[i]) : 0u;
    }
    float top = 0.0f, mine = 0.0f, sum = 0.0f;   // lane j holds the j-th chosen
    uint32_t taken = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (!(taken >> i & 1) && lane + 32 * i < n && (at == 0x7fffffff || key[i] > best)) {
                best = key[i];
                at = lane + 32 * i;
            }
        const uint32_t most = __reduce_max_sync(0xffffffffu, at == 0x7fffffff ? 0u : best);
        at = __reduce_min_sync(0xffffffffu, at != 0x7fffffff && best == most ? at : 0x7fffffff);
        if ((at & 31) == lane) taken |= 1u << (at >> 5);
        const float v = value_of(most);
        if (j == 0) top = v;
        const float e = expf(v - top);
        if (norm) sum += e;
        if (lane == j) mine = e;
        if (lane == 0) ids[j] = at;
    }
    if (!norm) {
#pragma unroll
        for (int i = 0; i < NE; ++i) sum += lane + 32 * i < n ? expf(l[i] - top) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < k) gate[lane] = mine / sum * scale;
}

// The router: logits x R^T in fp32 (a lane's products in four running sums),
// then the choice.  A cluster of CTAs takes TT tokens and shares out the
// experts, a warp per expert (or several, by columns, where there are fewer
// experts than warps); its logits meet in shared memory and CTA t chooses for
// token t.  Latency bounds it: the tokens go through shared memory, so that a
// lane has four loads of the router in flight at a time (eight would leave room
// for one CTA on an SM, and 61 tokens in two waves).  In one launch: a
// first version that left the choice to every CTA of the next kernel added 5 us
// there for 61 tokens of 128 experts.
constexpr int kRouteCluster = 8, kRouteWarps = 16, kRouteCols = 2048;   // columns of the tokens in shared memory at a time

template <int TT>
__global__ void __launch_bounds__(kRouteWarps * 32, 2) route_kernel(const float* __restrict__ x, const float* __restrict__ router,
                                                                 int64_t cols, int n_tok, int n_exp, int k, bool norm, float scale,
                                                                 int32_t* __restrict__ ids, float* __restrict__ gate) {
    constexpr int kPer = QK_MOE_MAX_EXP / kRouteCluster;
    __shared__ float logits[TT][kPer], parts[kPer][TT];   // [expert's part] where warps share a row
    __shared__ __align__(16) float xs[TT * kRouteCols];
    cg::cluster_group cl = cg::this_cluster();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = (int)cl.block_rank();
    const int t0 = (int)(blockIdx.x / kRouteCluster) * TT, width = (int)cols;
    const int per = (n_exp + kRouteCluster - 1) / kRouteCluster, e0 = rank * per, mine = max(0, min(per, n_exp - e0));
    // Fewer experts than warps: several warps to a row of the router.
    const int share = per >= kRouteWarps ? 1 : kRouteWarps / per, part = warp % share;
    const bool on = warp < kRouteWarps / share * share;
    pdl_launch_dependents();
    pdl_wait_prior();   // x
    for (int i = threadIdx.x; i < kPer * TT; i += kRouteWarps * 32) (&parts[0][0])[i] = 0.0f;
    for (int base = 0; base < width; base += kRouteCols) {
        const int n = min(kRouteCols, width - base);
        __syncthreads();   // all are done with the columns before
        for (int i = threadIdx.x; i < TT * (n / 4); i += kRouteWarps * 32) {
            const int t = i / (n / 4), c = 4 * (i - t * (n / 4));
            cp_async16(&xs[t * kRouteCols + c], x + (int64_t)min(t0 + t, n_tok - 1) * cols + base + c);
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        for (int e = warp / share; e < mine && on; e += kRouteWarps / share) {
            float4 acc[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float* w = router + (int64_t)(e0 + e) * cols + base;
            const int c0 = lane * 4 + part * 128, steps = c0 < n ? (n - 1 - c0) / (128 * share) + 1 : 0;
#pragma unroll 4
            for (int i = 0; i < steps; ++i) {
                const int c = c0 + i * 128 * share;
                const float4 r = __ldg(reinterpret_cast<const float4*>(w + c));
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const float4 v = *reinterpret_cast<const float4*>(&xs[t * kRouteCols + c]);
                    acc[t].x = fmaf(r.x, v.x, acc[t].x);
                    acc[t].y = fmaf(r.y, v.y, acc[t].y);
                    acc[t].z = fmaf(r.z, v.z, acc[t].z);
                    acc[t].w = fmaf(r.w, v.w, acc[t].w);
                }
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                float v = (acc[t].x + acc[t].y) + (acc[t].z + acc[t].w);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) parts[e * share + part][t] += v;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < mine * TT; i += kRouteWarps * 32) {
        const int e = i / TT, t = i - e * TT;
        float v = 0.0f;
        for (int q = 0; q < share; ++q) v += parts[e * share + q][t];
        logits[t][e] = v;
    }
    cl.sync();
    for (int t = rank; t < TT; t += kRouteCluster) {
        const int tok = t0 + t;
        if (warp != 0 || tok >= n_tok) continue;
        auto logit = [&](int e) { return cl.map_shared_rank(&logits[t][0], e / per)[e % per]; };
        int32_t* io = ids + (int64_t)tok * k;
        float* go = gate + (int64_t)tok * k;
        if (n_exp <= 128) choose<4>(logit, n_exp, k, norm, scale, lane, io, go);
        else if (n_exp <= 256) choose<8>(logit, n_exp, k, norm, scale, lane, io, go);
        else choose<16>(logit, n_exp, k, norm, scale, lane, io, go);
    }
    cl.sync();   // nobody leaves while its logits are read
}

template <int TT>
static cudaError_t route(const MoeArgs& m, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((m.n_tok + TT - 1) / TT * kRouteCluster));
    cfg.blockDim = dim3(kRouteWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kRouteCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, route_kernel<TT>, m.x, m.router, m.cols, m.n_tok, m.n_exp, m.k, m.norm, m.scale, m.ids, m.gate);
}

// out[tok] = sum over the token's experts of gate * y, y the slices' sums added
// in order.  A thread per expert and four columns, so that all loads are in
// flight at once (they come from L2); the experts are then added in order.
constexpr int kSumCols = 32;   // threads' columns of a CTA, four each
__global__ void __launch_bounds__(kSumCols * QK_MOE_MAX_K) sum_kernel(const float* __restrict__ y, const int32_t* __restrict__ ids,
                                                                      const float* __restrict__ gate, int n_exp, int n_tok, int k,
                                                                      int64_t cols, int slices, float* __restrict__ out) {
    __shared__ float4 part[QK_MOE_MAX_K][kSumCols];
    const int64_t c = ((int64_t)blockIdx.x * kSumCols + threadIdx.x) * 4;
    const int tok = blockIdx.y, j = threadIdx.y, pair = tok * k + j;
    pdl_launch_dependents();
    pdl_wait_prior();
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int e = __ldcg(ids + pair);
    if (c < cols && e >= 0 && e < n_exp) {   // (nothing was written for a pair without an expert)
        const float g = __ldcg(gate + pair);
        const float4* src = reinterpret_cast<const float4*>(y + (int64_t)pair * cols + c);
        const int64_t slice = (int64_t)n_tok * k * cols / 4;
#pragma unroll 4
        for (int s = 0; s < slices; ++s) {
            const float4 w = __ldcg(src + s * slice);
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        v.x *= g, v.y *= g, v.z *= g, v.w *= g;
    }
    part[j][threadIdx.x] = v;
    __syncthreads();
    if (j != 0 || c >= cols) return;
    for (int q = 1; q < k; ++q) {
        const float4 w = part[q][threadIdx.x];
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    float* o = out + (int64_t)tok * cols + c;   // 4-byte aligned
    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
}

}  // namespace moe

// The arguments of the two products and their workspace: the sums of `up`, then
// those of `down`.
static cudaError_t set_up(const MoeArgs& m, int sms, moe::Args& up, moe::Args& down, int64_t* bytes) {
    up = moe::Args{};
    up.cols = m.cols;
    up.rows = m.rows;
    up.n_exp = m.n_exp;
    up.n_tok = m.n_tok;
    up.k = m.k;
    up.pairs = m.n_tok * m.k;
    down = up;
    down.cols = m.rows;
    down.rows = m.cols;
    cudaError_t e = moe::launch_up(m.type, up, sms, nullptr, false);
    if (e == cudaSuccess) e = moe::launch_down(m.type_down, down, sms, nullptr, false);
    if (e != cudaSuccess) return e;
    bytes[0] = (int64_t)2 * up.slices * up.pairs * m.rows * 4;
    bytes[1] = (int64_t)down.slices * up.pairs * m.cols * 4;
    return e;
}

int64_t moe_ws_bytes(const MoeArgs& m, int sms) {
    moe::Args up, down;
    int64_t bytes[2];
    return set_up(m, sms, up, down, bytes) == cudaSuccess ? bytes[0] + bytes[1] : 0;
}

int moe_group(const MoeArgs& m, bool down_product, int sms) {
    moe::Args up, down;
    int64_t bytes[2];
    return set_up(m, sms, up, down, bytes) == cudaSuccess ? (down_product ? down.cap : up.cap) : 0;
}

cudaError_t launch_moe_ffn(const MoeArgs& m, unsigned* status, int sms, cudaStream_t s) {
    moe::Args up, down;
    int64_t bytes[2];
    cudaError_t e = set_up(m, sms, up, down, bytes);
    if (e != cudaSuccess) return e;
    float* sums = static_cast<float*>(m.ws);
    float* y = sums + bytes[0] / 4;
    if (m.router) {
        e = m.n_tok == 1 ? moe::route<1>(m, s) : moe::route<4>(m, s);
        if (e != cudaSuccess) return e;
    }
    up.x = m.x;
    up.W0 = static_cast<const uint8_t*>(m.Wg);
    up.W1 = static_cast<const uint8_t*>(m.Wu);
    up.out = sums;
    down.x = sums;
    down.slices_in = up.slices;
    down.W0 = down.W1 = static_cast<const uint8_t*>(m.Wd);
    down.out = y;
    up.ids = down.ids = m.ids;
    up.status = down.status = status;
    e = moe::launch_up(m.type, up, sms, s, true);
    if (e == cudaSuccess) e = moe::launch_down(m.type_down, down, sms, s, true);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((m.cols / 4 + moe::kSumCols - 1) / moe::kSumCols), (unsigned)m.n_tok);
    cfg.blockDim = dim3(moe::kSumCols, (unsigned)m.k);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe::sum_kernel, (const float*)y, (const int32_t*)m.ids, (const float*)m.gate, m.n_exp, m.n_tok,
                              m.k, m.cols, down.slices, m.out);
}

}  // namespace qk
