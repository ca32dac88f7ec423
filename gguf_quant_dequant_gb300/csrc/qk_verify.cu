// qk_verify.cu -- drafted trees judged against the target's probabilities
// (qk_verify_tree).
//
// Weights of a row: e_v = exp((x_v - max x) / T), T the request's
// temperature; sums and thresholds in 64 bits.  From the root on, a node's
// children are tried in order: child c with token y is taken when
//   u_c q(y) S < W(y),   S = sum_v W_v,
// where without the drafter's probabilities q = 1 and W is e without the
// tokens refused before, and with them q is the drafter's row of the node and
// W_v = max(e_v - tau q_v, 0), tau the sum of the S of the refusals before.
// (The target's p after refusals is W / S: the usual residual max(p - q, 0),
// normed, written without norming.)  Where no child is taken the token after
// the path is the first v with sum_{v' <= v} W_v' > u S.  Only rows on the path
// are read, which is why the walk is one launch and not a pass over all rows.
//
// One cluster of CTAs walks one request: every CTA has a contiguous part of
// the vocabulary, every warp a contiguous part of that, so that the warps'
// sums in order bracket the threshold and one warp looks its part up again.
// All CTAs hold all warps' sums (written through distributed shared memory)
// and take every decision alike.
#include <algorithm>
#include <cooperative_groups.h>

#include "qk_internal.h"
#include "qk_ptx.cuh"

namespace cg = cooperative_groups;

namespace qk {
namespace vt {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kMaxCluster = 16;
constexpr int kNodes = QK_TREE_MAX;
constexpr float kGreedy = 0x1p-20f;   // temperatures below it: the largest logit

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, int64_t v) {
    return BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(row)[v] << 16) : static_cast<const float*>(row)[v];
}

// exp((x - top) rate) for the largest logit top of the row; NaN counts as -inf, and of a row with +inf only those count.
__device__ __forceinline__ float weight(float x, float top, float rate) {
    const float d = __fsub_rn(x, top);
    const float e = expf(__fmul_rn(d, rate));
    return x == top ? 1.0f : d > -INFINITY ? e : 0.0f;
}
__device__ __forceinline__ float rest(float e, float tau, float q) { return fmaxf(__fsub_rn(e, __fmul_rn(tau, q)), 0.0f); }

// Sum of fp32 values to about 2^-48: the running sum and the rounding it loses.
struct Sum {
    float h = 0.0f, l = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float s = __fadd_rn(h, v), b = __fsub_rn(s, h);
        l = __fadd_rn(l, __fadd_rn(__fsub_rn(h, __fsub_rn(s, b)), __fsub_rn(v, b)));
        h = s;
    }
    __device__ __forceinline__ double value() const { return (double)h + (double)l; }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Shared {
    double sums[2][kMaxCluster * kWarps];   // W's sum of every warp of the cluster; by turns
    double plain[kMaxCluster * kWarps];     // e's, of the current node
    float top[2][kMaxCluster];              // the largest logit of every CTA's part, and its place; by turns
    int best[2][kMaxCluster];
    float wtop[kWarps];
    int wbest[kWarps];
    int parent[kNodes], token[kNodes];
    int refused[kNodes];                    // tokens taken out of the current node's W
    int n_refused, verdict, child, part, usual;
    double total, before, target;
};
enum : int { kNone = 0, kTaken = 1, kRefused = 2 };   // of the children from one on

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t r = blockIdx.x / C;
    int64_t row0 = a.cu[r], row1 = a.cu[r + 1];
    row0 = min(max(row0, (int64_t)0), a.n_rows);
    row1 = min(max(row1, row0), a.n_rows);
    const int n = (int)min(row1 - row0, (int64_t)kNodes);
    int32_t* path = a.path + r * a.path_stride;
    int32_t* tokens = a.tokens + r * a.path_stride;
    if (rank == 0)
        for (int64_t i = tid; i < a.path_stride; i += kThreads) path[i] = tokens[i] = -1;
    if (n == 0) {
        if (rank == 0 && tid == 0) a.n_path[r] = 0;
        return;   // the whole cluster
    }
    const float temp = a.temp[r];
    const bool greedy = !(temp >= kGreedy);
    const float rate = greedy ? 1.0f : __frcp_rn(temp);
    const bool drafter = a.probs != nullptr && !greedy;
    if (tid < n) {
        // the parent is the nearest ancestor: the highest bit below the node's own
        const uint64_t up = a.mask ? a.mask[row0 + tid] & ((1ull << tid) - 1) : (tid ? 1ull << (tid - 1) : 0ull);
        sh.parent[tid] = up ? 63 - __clzll((long long)up) : -1;
        sh.token[tid] = a.draft ? a.draft[row0 + tid] : -1;
    }
    // My part of the vocabulary: v0 .. v1 - 1, a multiple of a warp's step long (but the last).
    constexpr int kVec = VEC ? (BF16 ? 8 : 4) : 1, kStep = 32 * kVec;
    const int64_t share = ((a.vocab + (int64_t)C * kWarps - 1) / ((int64_t)C * kWarps) + kStep - 1) / kStep * kStep;
    const int64_t v0 = min((int64_t)(rank * kWarps + warp) * share, a.vocab), v1 = min(v0 + share, a.vocab);
    // f(v, x) for the elements of the warp's part, in a lane's order
    auto walk = [&](const void* row, auto f) {
        for (int64_t v = v0 + lane * kVec; v < v1; v += kStep) {
            if (VEC && v + kVec <= v1) {
                float x[kVec];
                if constexpr (BF16) {
                    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + v);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < kVec; ++i) x[i] = __uint_as_float(i & 1 ? w[(i >> 1) & 3] & 0xffff0000u : w[(i >> 1) & 3] << 16);
                } else {
                    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + v);
                    const float w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < kVec; ++i) x[i] = w[i & 3];
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) f(v + i, x[i]);
            } else {
                for (int i = 0; i < kVec && v + i < v1; ++i) f(v + i, logit<BF16>(row, v + i));
            }
        }
    };
    // An exchange writes one buffer and ends with the cluster's barrier; the buffer is written again two exchanges of its
    // kind later, after another barrier that every CTA reaches only when it has read it.
    int top_turn = 0, sum_turn = 0;
    // Every warp's sum to every CTA of the cluster, and their sum in order.
    auto exchange = [&](double mine, bool plain) {
        sum_turn ^= 1;
        if (lane < C) cl.map_shared_rank(&sh, lane)->sums[sum_turn][rank * kWarps + warp] = mine;
        cl.sync();
        if (warp == 0) {
            double s = 0.0;
            for (int i = lane; i < C * kWarps; i += 32) {
                const double v = sh.sums[sum_turn][i];
                if (plain) sh.plain[i] = v;
                s += v;
            }
            s = warp_sum(s);
            if (lane == 0) sh.total = s;
        }
        __syncthreads();
    };
    int cur = 0, length = 1;
    if (rank == 0 && tid == 0) path[0] = 0;
    cl.sync();   // every CTA of the cluster runs before another writes to its shared memory
    for (;;) {
        const void* row = static_cast<const uint8_t*>(a.logits) + (row0 + cur) * a.row_stride * (BF16 ? 2 : 4);
        const float* q = drafter ? a.probs + (row0 + cur) * a.probs_stride : nullptr;
        // The row's largest logit and its first place.
        float m = -INFINITY;
        int at = 0x7fffffff;
        walk(row, [&](int64_t v, float x) {
            if (x > m) {
                m = x;
                at = (int)v;
            }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, m, o);
            const int oa = __shfl_xor_sync(0xffffffffu, at, o);
            if (om > m || (om == m && oa < at)) {
                m = om;
                at = oa;
            }
        }
        if (lane == 0) {
            sh.wtop[warp] = m;
            sh.wbest[warp] = at;
        }
        __syncthreads();
        if (warp == 0) {
            m = lane < kWarps ? sh.wtop[lane] : -INFINITY;
            at = lane < kWarps ? sh.wbest[lane] : 0x7fffffff;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float om = __shfl_xor_sync(0xffffffffu, m, o);
                const int oa = __shfl_xor_sync(0xffffffffu, at, o);
                if (om > m || (om == m && oa < at)) {
                    m = om;
                    at = oa;
                }
            }
            if (lane < C) {
                Shared* p = cl.map_shared_rank(&sh, lane);
                p->top[top_turn][rank] = m;
                p->best[top_turn][rank] = at;
            }
        }
        cl.sync();
        m = -INFINITY;
        at = 0x7fffffff;
        for (int c = 0; c < C; ++c)
            if (sh.top[top_turn][c] > m) {   // parts in order: the first place stays
                m = sh.top[top_turn][c];
                at = sh.best[top_turn][c];
            }
        const float top = m;
        const int best = at;   // 0x7fffffff: a row with nothing above -inf
        top_turn ^= 1;
        if (greedy) {
            if (warp == 0) {
                int next = 0x7fffffff;
                for (int i = lane; i < n; i += 32)
                    if (sh.parent[i] == cur && sh.token[i] == best) next = min(next, i);
                next = __reduce_min_sync(0xffffffffu, next);
                if (lane == 0) sh.child = next == 0x7fffffff || length >= a.path_stride ? -1 : next;
            }
            __syncthreads();
            const int next = sh.child;
            __syncthreads();
            if (next < 0) {
                if (rank == 0 && tid == 0) {
                    tokens[length - 1] = best == 0x7fffffff ? -1 : best;
                    a.n_path[r] = length;
                }
                break;
            }
            if (rank == 0 && tid == 0) {
                tokens[length - 1] = sh.token[next];
                path[length] = next;
            }
            cur = next;
            ++length;
            continue;
        }
        // The row's sum.
        {
            Sum s;
            if (top > -INFINITY) walk(row, [&](int64_t, float x) { s.add(weight(x, top, rate)); });
            if (tid == 0) sh.n_refused = 0;
            exchange(warp_sum(s.value()), true);
        }
        // The children, in order: all of them at once, or with the drafter's probabilities one by one, as a refusal
        // changes every W.
        int verdict = kNone, first = cur + 1;
        double tau = 0.0;
        while (length < a.path_stride) {
            if (warp == 0) {
                int got = kNone, which = n;
                for (int base = first & ~31; base < n && got == kNone; base += 32) {
                    const int i = base + lane;
                    const bool child = i >= first && i < n && sh.parent[i] == cur;
                    const int y = child ? sh.token[i] : -1;
                    float w = 0.0f, qy = 1.0f, u = 0.0f;
                    if (y >= 0 && y < a.vocab && top > -INFINITY) {
                        w = weight(logit<BF16>(row, y), top, rate);
                        if (drafter) {
                            qy = q[y];
                            if (tau > 0.0) w = rest(w, (float)tau, qy);
                        }
                        u = a.u_accept[row0 + i];
                    }
                    unsigned todo = __ballot_sync(0xffffffffu, child);
                    while (todo) {
                        const int c = __ffs(todo) - 1;
                        todo &= todo - 1;
                        const int yc = __shfl_sync(0xffffffffu, y, c);
                        float wc = __shfl_sync(0xffffffffu, w, c);
                        const float qc = __shfl_sync(0xffffffffu, qy, c), uc = __shfl_sync(0xffffffffu, u, c);
                        if (!drafter) {
                            bool gone = false;
                            for (int k = lane; k < sh.n_refused; k += 32) gone |= sh.refused[k] == yc;
                            if (__any_sync(0xffffffffu, gone)) wc = 0.0f;
                        }
                        const double S = sh.total;
                        __syncwarp();
                        which = base + c;
                        if ((double)uc * (double)qc * S < (double)wc) {
                            got = kTaken;
                            break;
                        }
                        if (drafter) {
                            got = kRefused;
                            break;
                        }
                        if (wc > 0.0f && lane == 0) {
                            sh.refused[sh.n_refused++] = yc;
                            const int64_t part = yc / share;   // the warp whose part it is
                            const double v = sh.sums[sum_turn][part], left = v - (double)wc;
                            sh.sums[sum_turn][part] = left > 1e-13 * v ? left : 0.0;   // what rounding leaves of nothing
                            sh.total = S - (double)wc;
                        }
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    sh.verdict = got;
                    sh.child = which;
                }
            }
            __syncthreads();
            verdict = sh.verdict;
            first = sh.child;
            const double S = sh.total;
            if (verdict != kRefused) break;
            ++first;
            tau += S;
            Sum s;
            const float off = (float)tau;
            if (top > -INFINITY) walk(row, [&](int64_t v, float x) { s.add(rest(weight(x, top, rate), off, q[v])); });
            exchange(warp_sum(s.value()), false);   // (its barriers also part this round's verdict from the next)
        }
        if (verdict == kTaken) {
            if (rank == 0 && tid == 0) {
                tokens[length - 1] = sh.token[first];
                path[length] = first;
            }
            cur = first;
            ++length;
            continue;
        }
        // The token after the path: the warp whose part holds the threshold, then the token in it.
        if (warp == 0) {
            const bool usual = sh.total > 0.0;   // nothing left (by rounding): the row's own weights
            const double* part = usual ? sh.sums[sum_turn] : sh.plain;
            const int parts = C * kWarps, each = (parts + 31) / 32;
            double mine = 0.0;
            for (int k = 0; k < each; ++k)
                if (lane * each + k < parts) mine += part[lane * each + k];
            double upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double t = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += t;
            }
            const double S = __shfl_sync(0xffffffffu, upto, 31);
            const double target = (double)a.u_sample[r] * S;
            double run = upto - mine, before = 0.0;
            int hit = 0x7fffffff, last = -1;
            for (int k = 0; k < each; ++k) {
                const int i = lane * each + k;
                if (i < parts && part[i] > 0.0) {
                    last = i;
                    if (hit == 0x7fffffff && run + part[i] > target) {
                        hit = i;
                        before = run;
                    }
                    run += part[i];
                }
            }
            const int found = __reduce_min_sync(0xffffffffu, hit);
            last = __reduce_max_sync(0xffffffffu, last);
            if (lane == 0) {
                sh.part = found != 0x7fffffff ? found : last;   // none when rounding puts the threshold at the end: the last token
                sh.target = found != 0x7fffffff ? target : INFINITY;
                sh.before = 0.0;
                sh.usual = usual;
            }
            __syncwarp();
            if (found != 0x7fffffff && hit == found) sh.before = before;
        }
        __syncthreads();
        const int part = sh.part;
        if (part < 0) {   // a row without weight
            if (rank == 0 && tid == 0) a.n_path[r] = length;
            break;
        }
        if (part / kWarps == rank && part % kWarps == warp) {
            const bool usual = sh.usual != 0;
            const double target = sh.target;
            const float off = (float)tau;
            double run = sh.before;
            int token = -1, last = -1;
            for (int64_t b = v0; b < v1 && token < 0; b += kStep) {
                double w[kVec], mine = 0.0;
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const int64_t v = b + lane * kVec + i;
                    float e = v < v1 ? weight(logit<BF16>(row, v), top, rate) : 0.0f;
                    if (usual && drafter && tau > 0.0 && v < v1) e = rest(e, off, q[v]);
                    if (usual && !drafter)
                        for (int k = 0; k < sh.n_refused; ++k)
                            if (sh.refused[k] == v) e = 0.0f;
                    w[i] = e;
                    mine += w[i];
                }
                double upto = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double t = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += t;
                }
                double at = run + (upto - mine);
                int hit = 0x7fffffff, some = -1;
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (w[i] > 0.0) {
                        at += w[i];
                        some = (int)(b + lane * kVec + i);
                        if (hit == 0x7fffffff && at > target) hit = some;
                    }
                hit = __reduce_min_sync(0xffffffffu, hit);
                last = max(last, __reduce_max_sync(0xffffffffu, some));
                if (hit != 0x7fffffff) token = hit;
                run += __shfl_sync(0xffffffffu, upto, 31);
            }
            if (lane == 0) {
                tokens[length - 1] = token >= 0 ? token : last;
                a.n_path[r] = length;
            }
        }
        break;
    }
}

template <bool BF16, bool VEC>
static cudaError_t go(const VerifyArgs& a, int cluster, cudaStream_t s) {
    auto kern = verify_kernel<BF16, VEC>;
    if (cluster > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n_req * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace vt

cudaError_t launch_verify_tree(const VerifyArgs& a, int sms, cudaStream_t s) {
    // CTAs of a request: as many as leave each some thousand tokens and all of them a place at once.
    int cluster = 8;
    while (cluster > 1 && ((int64_t)cluster * a.n_req > 2 * sms || a.vocab / cluster < 1024)) cluster >>= 1;
    const int es = a.bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.row_stride * es % 16 == 0;
    if (a.bf16) return vec ? vt::go<true, true>(a, cluster, s) : vt::go<true, false>(a, cluster, s);
    return vec ? vt::go<false, true>(a, cluster, s) : vt::go<false, false>(a, cluster, s);
}

}  // namespace qk
