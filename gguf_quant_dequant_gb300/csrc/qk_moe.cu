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

static int64_t logits_bytes(int n_tok, int n_exp) { return ((int64_t)n_tok * n_exp * 4 + 15) & ~(int64_t)15; }

}  // namespace moe

int64_t moe_ws_bytes(int n_tok, int k, int n_exp, int64_t rows) {
    return moe::logits_bytes(n_tok, n_exp) + (int64_t)n_tok * k * rows * 4;
}

cudaError_t launch_moe_ffn(const MoeArgs& m, unsigned* status, int sms, cudaStream_t s) {
    float* logits = static_cast<float*>(m.ws);
    float* h = logits + moe::logits_bytes(m.n_tok, m.n_exp) / 4;
    if (m.router) {
        const cudaError_t e = m.n_tok == 1 ? moe::route<1>(m.x, m.router, m.cols, m.n_tok, m.n_exp, logits, s)
                                           : moe::route<8>(m.x, m.router, m.cols, m.n_tok, m.n_exp, logits, s);
        if (e != cudaSuccess) return e;
    }
    moe::Args a{};
    a.x = m.x;
    a.cols = m.cols;
    a.rows = m.rows;
    a.W0 = static_cast<const uint8_t*>(m.Wg);
    a.W1 = static_cast<const uint8_t*>(m.Wu);
    a.n_exp = m.n_exp;
    a.n_tok = m.n_tok;
    a.k = m.k;
    a.pairs = m.n_tok * m.k;
    a.logits = m.router ? logits : nullptr;
    a.norm = m.norm;
    a.scale = m.scale;
    a.ids = m.ids;
    a.gate = m.gate;
    a.out = h;
    a.status = status;
    moe::Args b = a;
    const cudaError_t e = moe::launch_up(m.type, a, sms, s);
    if (e != cudaSuccess) return e;
    b.x = h;
    b.cols = m.rows;
    b.rows = m.cols;
    b.W0 = static_cast<const uint8_t*>(m.Wd);
    b.W1 = nullptr;
    b.logits = nullptr;
    b.out = m.out;
    return moe::launch_down(m.type_down, b, sms, s);
}

}  // namespace qk
