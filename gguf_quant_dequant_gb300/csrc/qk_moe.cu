// qk_moe.cu -- a mixture-of-experts layer (qk_moe_ffn): the router's logits,
// and the launches of the layer.
#include "qk_internal.h"
#include "qk_moe.cuh"

namespace qk {
namespace moe {

// Router logits [n_tok, n_exp] = x R^T in fp32: a warp per expert and TT
// tokens, a lane's products in four running sums.  The matrix is read once per
// TT tokens (L2 serves the repeats); a megabyte of it, so latency bounds it.
constexpr int kRouteWarps = 4;

template <int TT>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const float* __restrict__ x, const float* __restrict__ router,
                                                                 int64_t cols, int n_tok, int n_exp, float* __restrict__ logits) {
    const int lane = threadIdx.x & 31, e = blockIdx.x * kRouteWarps + (threadIdx.x >> 5), t0 = blockIdx.y * TT;
    pdl_launch_dependents();
    pdl_wait_prior();   // x
    if (e >= n_exp) return;
    float4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* w = router + (int64_t)e * cols;
#pragma unroll 4
    for (int64_t c = lane * 4; c < cols; c += 128) {
        const float4 r = *reinterpret_cast<const float4*>(w + c);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float4 v = *reinterpret_cast<const float4*>(x + (int64_t)min(t0 + t, n_tok - 1) * cols + c);
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
        if (lane == 0 && t0 + t < n_tok) logits[(int64_t)(t0 + t) * n_exp + e] = v;
    }
}

template <int TT>
static cudaError_t route(const float* x, const float* router, int64_t cols, int n_tok, int n_exp, float* logits, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((n_exp + kRouteWarps - 1) / kRouteWarps), (unsigned)((n_tok + TT - 1) / TT));
    cfg.blockDim = dim3(kRouteWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_kernel<TT>, x, router, cols, n_tok, n_exp, logits);
}

// out[tok] = sum over the token's experts of gate * y, y the slices' sums added
// in order.  Everything comes from L2: 61 tokens of 8 experts of 2048 rows read
// 4 MB.
constexpr int kSumThreads = 128;
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const float* __restrict__ y, const int32_t* __restrict__ ids,
                                                          const float* __restrict__ gate, int n_exp, int n_tok, int k, int64_t cols,
                                                          int slices, float* __restrict__ out) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const int64_t c = ((int64_t)blockIdx.x * kSumThreads + threadIdx.x) * 4;
    const int tok = blockIdx.y;
    if (c >= cols) return;
    const int64_t slice = (int64_t)n_tok * k * cols;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int j = 0; j < k; ++j) {
        const int pair = tok * k + j, e = __ldcg(ids + pair);
        if (e < 0 || e >= n_exp) continue;   // nothing was written for it
        const float g = __ldcg(gate + pair);
        const float* src = y + (int64_t)pair * cols + c;
        float4 v = __ldcg(reinterpret_cast<const float4*>(src));
        for (int s = 1; s < slices; ++s) {
            const float4 w = __ldcg(reinterpret_cast<const float4*>(src + s * slice));
            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        acc.x += g * v.x, acc.y += g * v.y, acc.z += g * v.z, acc.w += g * v.w;
    }
    float* o = out + (int64_t)tok * cols + c;   // 4-byte aligned
    o[0] = acc.x, o[1] = acc.y, o[2] = acc.z, o[3] = acc.w;
}

static int64_t logits_bytes(int n_tok, int n_exp) { return ((int64_t)n_tok * n_exp * 4 + 15) & ~(int64_t)15; }

}  // namespace moe

// The arguments of the two products and their workspace: the router's logits,
// the sums of `up`, those of `down`.
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
    bytes[0] = moe::logits_bytes(m.n_tok, m.n_exp);
    bytes[1] = (int64_t)2 * up.slices * up.pairs * m.rows * 4;
    bytes[2] = (int64_t)down.slices * up.pairs * m.cols * 4;
    return e;
}

int64_t moe_ws_bytes(const MoeArgs& m, int sms) {
    moe::Args up, down;
    int64_t bytes[3];
    return set_up(m, sms, up, down, bytes) == cudaSuccess ? bytes[0] + bytes[1] + bytes[2] : 0;
}

cudaError_t launch_moe_ffn(const MoeArgs& m, unsigned* status, int sms, cudaStream_t s) {
    moe::Args up, down;
    int64_t bytes[3];
    cudaError_t e = set_up(m, sms, up, down, bytes);
    if (e != cudaSuccess) return e;
    float* logits = static_cast<float*>(m.ws);
    float* sums = logits + bytes[0] / 4;
    float* y = sums + bytes[1] / 4;
    if (m.router) {
        e = m.n_tok == 1 ? moe::route<1>(m.x, m.router, m.cols, m.n_tok, m.n_exp, logits, s)
                         : moe::route<8>(m.x, m.router, m.cols, m.n_tok, m.n_exp, logits, s);
        if (e != cudaSuccess) return e;
    }
    up.x = m.x;
    up.W0 = static_cast<const uint8_t*>(m.Wg);
    up.W1 = static_cast<const uint8_t*>(m.Wu);
    up.logits = m.router ? logits : nullptr;
    up.norm = m.norm;
    up.scale = m.scale;
    up.out = sums;
    down.x = sums;
    down.slices_in = up.slices;
    down.W0 = down.W1 = static_cast<const uint8_t*>(m.Wd);
    down.out = y;
    up.ids = down.ids = m.ids;
    up.gate = down.gate = m.gate;
    up.status = down.status = status;
    e = moe::launch_up(m.type, up, sms, s, true);
    if (e == cudaSuccess) e = moe::launch_down(m.type_down, down, sms, s, true);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((m.cols / 4 + moe::kSumThreads - 1) / moe::kSumThreads), (unsigned)m.n_tok);
    cfg.blockDim = dim3(moe::kSumThreads);
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
