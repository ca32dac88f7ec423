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
// the path is the first v with sum_{v' <= v} W_v' > u S.
//
// One cluster of CTAs walks one request: every CTA has a contiguous part of the
// vocabulary, every warp a contiguous part of that, so that the warps' sums in
// order bracket the threshold and one part is looked through again.  A step of
// the walk is a chain of latencies (the row, its maximum over the cluster, its
// sum over the cluster: 5 us for one request, 12 us for 48), so:
//   * the rows that a walk without refusals would reach (the root, its first
//     child, that one's first child, ..) are summed beforehand, all at once, in
//     pieces of 1,024 logits, relative to the piece's largest.  A child that is
//     taken by a margin above what such a sum can be off is passed over without
//     going through its parent's row; everything else is decided by the walk's
//     exact sums, so the answer is the same with and without the pieces.  48
//     chains of 8 rows of 128,256 fp32: 128 us without, 72 us with them (39 us
//     of it the pieces', at 5.1 TB/s); one chain of 6 rows of 32,000: 21 and 13
//     us, of 64: 69 and 37; trees of 64 nodes: 35 either way;
//   * a thread keeps its logits of the row, then their weights, in registers
//     (up to kKeep of them; longer parts are read again from L2; kept in shared
//     memory they cost 15 % more than either);
//   * each warp writes its maximum and its sum to every CTA of the cluster: one
//     cluster barrier per exchange, and every CTA decides by itself;
//   * the next row of a chain is asked for (into L2) while the sum is formed.
#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>
#include <cstdint>

#include "qk_internal.h"
#include "qk_ptx.cuh"

namespace cg = cooperative_groups;

namespace qk {
namespace vt {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kPieceWarps = 8, kPieceCtas = 4;   // (CTAs on an SM)
constexpr int kNodes = QK_TREE_MAX;
constexpr int kKeep = 32;             // logits of a row that a thread keeps
constexpr float kGreedy = 0x1p-20f;   // temperatures below it: the largest logit

template <bool BF16>
__device__ __forceinline__ float logit(const void* row, int64_t v) {
    return BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(row)[v] << 16) : static_cast<const float*>(row)[v];
}

// exp((x - top) rate) for the largest logit top of the row, and its parts for
// two at a time: NaN counts as -inf (the maximum drops it; exp(-200) is 0).  A
// row with +inf is given top = FLT_MAX and rate 1, which leaves its mass there.
__device__ __forceinline__ float exponent(float t) { return fminf(fmaxf(t, -200.0f), 0.0f); }
__device__ __forceinline__ float weight(float x, float top, float rate) {
    return expf(exponent(__fmul_rn(__fsub_rn(x, top), rate)));
}
__device__ __forceinline__ float2 weight2(float2 x, float top, float rate) {
    const float2 t = __fmul2_rn(__fadd2_rn(x, make_float2(-top, -top)), make_float2(rate, rate));
    return make_float2(expf(exponent(t.x)), expf(exponent(t.y)));
}
__device__ __forceinline__ float rest(float e, float tau, float q) { return fmaxf(__fsub_rn(e, __fmul_rn(tau, q)), 0.0f); }

// Sums are of weights as whole numbers of 2^-bits, each rounded by itself (bits = 46 for up to 65,536 tokens, one less for
// each doubling), so that they are the same in whatever order and by whatever threads they are formed: a row's sum, its
// parts' sums and the running sum that finds a token agree to the last bit.  On this GPU a 64-bit floating addition costs a
// warp sixteen cycles of the whole SM, and two reductions with them took 2.9 us a row.
struct Fix {
    float up;      // 2^bits
    double down;   // 2^-bits
    float magic;   // 1.5 2^(23 - bits): added to a number below 2^-24, its last place is 2^-bits
    int high;      // bits - 23
    static __device__ __forceinline__ Fix unit(int bits) {
        return {__uint_as_float((uint32_t)(127 + bits) << 23), __longlong_as_double((int64_t)(1023 - bits) << 52),
                __uint_as_float(((uint32_t)(150 - bits) << 23) | 0x400000u), bits - 23};
    }
    __device__ __forceinline__ int64_t of(float v) const { return __float2ll_rn(v * up); }
};
// Running sum of `of` of weights in 0 .. 1 without a conversion each: v + 1 rounds v to 23 bits, which stand in the sum's
// mantissa as a whole number; what that leaves out, added to `magic`, does the same for the bits below.  (A tie is one of the
// low part alone, and both parts' offsets are even, so it falls as in `of`.)  Both mantissas are added as 32-bit words,
// offsets and all, which holds for 511 weights; two integer additions more for two weights than compensated fp32 sums.
struct Sum {
    uint32_t h = 0, l = 0;
    int n = 0;   // weights in them
    int64_t all = 0;
    __device__ __forceinline__ void add(float2 v, const Fix& f) {
        const float2 t = __fadd2_rn(v, make_float2(1.0f, 1.0f)), d = __fadd2_rn(t, make_float2(-1.0f, -1.0f));
        const float2 r = __fadd2_rn(__fadd2_rn(v, make_float2(-d.x, -d.y)), make_float2(f.magic, f.magic));
        h += __float_as_uint(t.x) + __float_as_uint(t.y);
        l += __float_as_uint(r.x) + __float_as_uint(r.y);
    }
    // kVec weights (one alone beside a zero).
    template <int N>
    __device__ __forceinline__ void add(const float (&v)[N], const Fix& f) {
        if constexpr (N == 1) {
            add(make_float2(v[0], 0.0f), f);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 2) add(make_float2(v[i], v[i + 1]), f);
        }
        n += N == 1 ? 2 : N;
    }
    __device__ __forceinline__ void flush(const Fix& f) {
        all += ((int64_t)(h - (uint32_t)n * 0x3f800000u) << f.high) + (int32_t)(l - (uint32_t)n * __float_as_uint(f.magic));
        h = l = 0;
        n = 0;
    }
    // Before up to 64 weights more.
    __device__ __forceinline__ void room(const Fix& f) {
        if (n > 511 - 64) flush(f);
    }
    __device__ __forceinline__ int64_t value(const Fix& f) {
        flush(f);
        return all;
    }
};
// Logits to weights.
template <int N>
__device__ __forceinline__ void weigh(float (&v)[N], float top, float rate) {
    if constexpr (N == 1) {
        v[0] = weight(v[0], top, rate);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 w = weight2(make_float2(v[i], v[i + 1]), top, rate);
            v[i] = w.x;
            v[i + 1] = w.y;
        }
    }
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}
// The largest of the warp's (m, at), the lowest place of equals.
__device__ __forceinline__ void warp_top(float& m, int& at) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, o);
        const int oa = __shfl_xor_sync(0xffffffffu, at, o);
        if (om > m || (om == m && oa < at)) {
            m = om;
            at = oa;
        }
    }
}

constexpr int kNowhere = 0x7fffffff;
struct Shared {
    int64_t sums[2][kMaxCluster * kWarps];  // W's sum of every warp of the cluster; by turns
    int64_t plain[kMaxCluster * kWarps];    // e's, of the last node, where a child was refused
    float top[2][kMaxCluster * kWarps];     // every warp's largest logit and its place; by turns
    int best[2][kMaxCluster * kWarps];
    int64_t piece[kWarps];                  // the sampled part's pieces
    int parent[kNodes], token[kNodes];
    int part, usual, next, again;
    float node_top[kNodes];                 // of the nodes' rows, where pieces were summed first: the largest logit, its place
    int node_best[kNodes], taken[kNodes];   // and the child that is taken for sure, or -1
    uint64_t refused;                       // children of the node, without the drafter's probabilities
    double tau;
    int64_t target, before;
};

// Elements of a warp's part: lane-wise vectors of kVec, 32 of them a step.
template <bool BF16, bool VEC>
struct Lanes {
    static constexpr int kVec = VEC ? (BF16 ? 8 : 4) : 1, kStep = 32 * kVec;
    // kVec logits from v on; -inf from v1 on (v < v1).
    static __device__ __forceinline__ void load(const void* row, int64_t v, int64_t v1, float (&x)[kVec]) {
        if (VEC && v + kVec <= v1) {
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
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) x[i] = v + i < v1 ? logit<BF16>(row, v + i) : -INFINITY;
        }
    }
};

// ------------------------------------------------------- rows at once --
// What is known of 1,024 of a row's logits: their largest and its first place,
// the sum of their weights relative to it, and the rate they were taken at.
struct Piece {
    float top;
    int best;
    float sum, rate;
};
constexpr int kPiece = 1024;
// How far the pieces' sum can be off the row's, and more.  Weights count down to
// exponents of -32 (2^31 of them come to less than 2^-15 of the largest's 1); up
// to there the fast exponential (2 + 1.2 |t| steps of 2^-23) and two roundings of
// the exponent (|t| 2^-23) leave less than a part 2^-16.  The row's own sum has
// every weight rounded to a whole number of its unit, at most 2^-15 of it in all
// up to kPieceVocab tokens.  A child is sure to be taken when it is by this margin.
constexpr double kSure = 1.0 + 0x1p-13;
constexpr int64_t kPieceVocab = 1 << 24;

// The parent of a request's node i (row `row` of the mask), or -1.
__device__ __forceinline__ int parent_of(const uint64_t* mask, int64_t row, int i) {
    // the nearest ancestor: the highest bit below the node's own
    const uint64_t up = mask ? mask[row] & ((1ull << i) - 1) : (i ? 1ull << (i - 1) : 0ull);
    return up ? 63 - __clzll((long long)up) : -1;
}
// The nodes that the walk reaches while no child is refused (the root, its first
// child, that one's first child, ..), by a warp; lane i has the parents of nodes
// i and i + 32.
__device__ __forceinline__ uint64_t first_line(int up0, int up1, int n, int lane) {
    uint64_t line = 1;
    for (int c = 0;;) {   // a parent is below its children: c rises
        const unsigned k0 = __ballot_sync(0xffffffffu, lane < n && up0 == c), k1 = __ballot_sync(0xffffffffu, lane + 32 < n && up1 == c);
        if (!(k0 | k1)) return line;
        c = k0 ? __ffs(k0) - 1 : 31 + __ffs(k1);
        line |= 1ull << c;
    }
}
// The k-th node of a line.
__device__ __forceinline__ int node_of(uint64_t line, int k) {
    for (; k > 0; --k) line &= line - 1;
    return __ffsll((long long)line) - 1;
}

// The rows of a request's first line, a piece a warp at a time; no warp waits for
// another's sums.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kPieceWarps * 32, kPieceCtas) piece_kernel(const VerifyArgs a, Piece* pieces, int per_row, int share) {
    using L = Lanes<BF16, VEC>;
    constexpr int kVec = L::kVec, kStep = L::kStep, kRegs = kPiece / kStep;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    const int64_t r = blockIdx.x / share;
    const int64_t row0 = min(max((int64_t)a.cu[r], (int64_t)0), a.n_rows), row1 = min(max((int64_t)a.cu[r + 1], row0), a.n_rows);
    const int n = (int)min(row1 - row0, (int64_t)kNodes);
    if (n < 2) return;
    const float temp = a.temp[r];
    const uint64_t line = first_line(lane < n ? parent_of(a.mask, row0 + lane, lane) : -1,
                                     lane + 32 < n ? parent_of(a.mask, row0 + lane + 32, lane + 32) : -1, n, lane);
    const bool greedy = !(temp >= kGreedy);
    const float rate = greedy ? 1.0f : __frcp_rn(temp);
    const int items = __popcll(line) * per_row;
    for (int i = (int)(blockIdx.x % share) * kPieceWarps + (threadIdx.x >> 5); i < items; i += share * kPieceWarps) {
        const int k = i / per_row, part = i - k * per_row;
        const int64_t row = row0 + node_of(line, k);
        const void* p = static_cast<const uint8_t*>(a.logits) + row * a.row_stride * (BF16 ? 2 : 4);
        const int64_t v0 = (int64_t)part * kPiece, v1 = min(v0 + kPiece, a.vocab);
        float x[kRegs][kVec];
#pragma unroll
        for (int k = 0; k < kRegs; ++k) {
            const int64_t v = v0 + k * kStep + lane * kVec;
            if (v < v1) {
                L::load(p, v, v1, x[k]);
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) x[k][i] = -INFINITY;
            }
        }
        float m = -INFINITY, total = 0.0f;
#pragma unroll
        for (int k = 0; k < kRegs; ++k)
#pragma unroll
            for (int i = 0; i < kVec; ++i) m = fmaxf(m, x[k][i]);
        int at = kNowhere;
        if (greedy) {
#pragma unroll
            for (int k = kRegs - 1; k >= 0; --k)
#pragma unroll
                for (int i = kVec - 1; i >= 0; --i)
                    if (x[k][i] == m && m > -INFINITY) at = (int)(v0 + k * kStep + lane * kVec + i);
            warp_top(m, at);
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (m > -INFINITY) {
                float s[4] = {0, 0, 0, 0};   // NaN stays: then nothing is sure
#pragma unroll
                for (int k = 0; k < kRegs; ++k)
#pragma unroll
                    for (int i = 0; i < kVec; ++i) s[(k * kVec + i) & 3] += __expf((x[k][i] - m) * rate);
                total = (s[0] + s[1]) + (s[2] + s[3]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        if (lane == 0) pieces[row * per_row + part] = Piece{m, at, total, rate};
    }
}

// KEEP: the part of a thread fits its registers.
template <bool BF16, bool VEC, bool KEEP>
__global__ void __launch_bounds__(kThreads, KEEP ? 1 : 2) verify_kernel(const VerifyArgs a, const Piece* pieces, int per_row) {
    using L = Lanes<BF16, VEC>;
    constexpr int kVec = L::kVec, kStep = L::kStep, kRegs = KEEP ? kKeep / kVec : 1, kAhead = KEEP ? 1 : 8 / (kVec > 4 ? 2 : 1);
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), parts = C * kWarps;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, me = rank * kWarps + warp;
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
        pdl_wait_prior();   // (no launch ends before the one that sums its pieces)
        return;   // the whole cluster
    }
    const float temp = a.temp[r], u_sample = a.u_sample[r];
    const bool greedy = !(temp >= kGreedy);
    const float rate_of = greedy ? 1.0f : __frcp_rn(temp);
    const bool drafter = a.probs != nullptr && !greedy;
    if (tid < n) {
        sh.parent[tid] = parent_of(a.mask, row0 + tid, tid);
        sh.token[tid] = a.draft[row0 + tid];
    }
    // My part of the vocabulary: v0 .. v1 - 1, a multiple of a step long (but the last).
    const int64_t share = ((a.vocab + parts - 1) / parts + kStep - 1) / kStep * kStep;
    const int64_t v0 = min(me * share, a.vocab), v1 = min(v0 + share, a.vocab);
    const Fix fix = Fix::unit(min(46, 62 - (32 - __clz((int)a.vocab - 1))));
    // An exchange writes one buffer and ends with the cluster's barrier; the buffer is written again two exchanges of its
    // kind later, after another barrier that every warp reaches only when it has read it.
    int top_turn = 0, sum_turn = 0;
    auto exchange = [&](int64_t mine) {   // every warp's sum to every CTA
        sum_turn ^= 1;
        if (lane < C) cl.map_shared_rank(&sh, lane)->sums[sum_turn][me] = mine;
        cl.sync();
    };
    auto total_of = [&]() {   // their sum
        int64_t s = 0;
        for (int i = lane; i < parts; i += 32) s += sh.sums[sum_turn][i];
        return warp_sum(s);
    };
    int cur = 0, length = 1;
    if (rank == 0 && tid == 0) path[0] = 0;
    cl.sync();   // every CTA of the cluster runs (and has its tree) before another writes to its shared memory
    pdl_wait_prior();   // the pieces
    uint64_t line = 0;   // the nodes whose rows were summed in pieces
    if (pieces && n > 1) {
        // A warp a node: its row's largest logit, and the child that is taken for sure once the node is reached, where the
        // pieces of the row decide by a margin (and no other child is tried before it).
        line = first_line(lane < n ? sh.parent[lane] : -1, lane + 32 < n ? sh.parent[lane + 32] : -1, n, lane);
        const int nodes = __popcll(line);
        for (int k = warp; k < nodes; k += kWarps) {
            const int p = node_of(line, k);
            const Piece* of = pieces + (row0 + p) * per_row;
            unsigned kids[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = lane + 32 * h;
                kids[h] = __ballot_sync(0xffffffffu, i > p && i < n && sh.parent[i] == p);
            }
            int c = kids[0] ? __ffs(kids[0]) - 1 : kids[1] ? 31 + __ffs(kids[1]) : -1;
            const int y = c >= 0 ? sh.token[c] : -1;
            const bool test = !greedy && y >= 0 && y < a.vocab;
            float x = 0.0f, qy = 1.0f, u = 0.0f;
            if (test) {
                x = logit<BF16>(static_cast<const uint8_t*>(a.logits) + (row0 + p) * a.row_stride * (BF16 ? 2 : 4), y);
                u = a.u_accept[row0 + c];
                if (drafter) qy = a.probs[(row0 + p) * a.probs_stride + y];
            }
            float m = -INFINITY;
            int at = kNowhere;
            bool same = true;
            // four loads of 16 bytes in flight a lane
            Piece some[4];
            auto four = [&](int base) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = base + 32 * j + lane;
                    some[j] = Piece{-INFINITY, kNowhere, 0.0f, rate_of};
                    if (i < per_row) {
                        const float4 u = *reinterpret_cast<const float4*>(of + i);
                        some[j] = Piece{u.x, __float_as_int(u.y), u.z, u.w};
                    }
                }
            };
            for (int base = 0; base < per_row; base += 128) {
                four(base);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    same &= some[j].rate == rate_of;
                    if (some[j].top > m) {
                        m = some[j].top;
                        at = some[j].best;
                    }
                }
            }
            warp_top(m, at);
            bool sure = false;
            if (greedy) {
#pragma unroll
                for (int h = 1; h >= 0; --h) {
                    const int i = lane + 32 * h;
                    const unsigned hit = __ballot_sync(0xffffffffu, (kids[h] >> lane & 1) && at != kNowhere && sh.token[i] == at);
                    if (hit) {
                        c = __ffs(hit) - 1 + 32 * h;
                        sure = true;
                    }
                }
            } else if (test && fabsf(m) < INFINITY) {
                double S = 0.0;
                for (int base = 0; base < per_row; base += 128) {
                    if (per_row > 128) four(base);
#pragma unroll
                    for (int j = 0; j < 4; ++j) S += (double)some[j].sum * (double)weight(some[j].top, m, rate_of);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
                sure = (double)u * (double)qy * S * kSure < (double)weight(x, m, rate_of);
            }
            sure = __all_sync(0xffffffffu, same) && sure;
            if (lane == 0) {
                sh.node_top[p] = m;
                sh.node_best[p] = at;
                sh.taken[p] = sure ? c : -1;
            }
        }
        __syncthreads();
    }
    for (;;) {
        while ((line >> cur & 1) && length < a.path_stride && sh.taken[cur] >= 0) {
            cur = sh.taken[cur];
            if (rank == 0 && tid == 0) {
                tokens[length - 1] = sh.token[cur];
                path[length] = cur;
            }
            ++length;
        }
        const void* row = static_cast<const uint8_t*>(a.logits) + (row0 + cur) * a.row_stride * (BF16 ? 2 : 4);
        const float* q = drafter ? a.probs + (row0 + cur) * a.probs_stride : nullptr;
        // The drafter's probabilities of kVec tokens from v on (0 behind the part: the weights there are 0 too).
        auto load_q = [&](int64_t v, float (&w)[kVec]) {
            if (kVec >= 4 && a.probs_vec && v + kVec <= v1) {
#pragma unroll
                for (int i = 0; i < kVec; i += 4) {
                    const float4 u = *reinterpret_cast<const float4*>(q + v + i);
                    w[i] = u.x;
                    if (kVec >= 4) w[(i + 1) % kVec] = u.y, w[(i + 2) % kVec] = u.z, w[(i + 3) % kVec] = u.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) w[i] = v + i < v1 ? q[v + i] : 0.0f;
            }
        };
        // My logits: kept, or passed by; the largest and its first place.
        float x[kRegs][kVec], m = -INFINITY;
        int at = kNowhere;
        auto look = [&](const float (&w)[kVec], int64_t v) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (w[i] > m) {
                    m = w[i];
                    at = (int)(v + i);
                }
        };
        if constexpr (KEEP) {
#pragma unroll
            for (int k = 0; k < kRegs; ++k) {
                const int64_t v = v0 + k * kStep + lane * kVec;
                if (v < v1) {
                    L::load(row, v, v1, x[k]);
                } else {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) x[k][i] = -INFINITY;
                }
            }
        }
        // What the tests of the children will read: lane i of a warp has child i, and i + 32.
        int kid[2];
        float kx[2], ku[2], kq[2];
        unsigned kids[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane + 32 * h;
            const bool child = i > cur && i < n && sh.parent[i] == cur;
            kids[h] = __ballot_sync(0xffffffffu, child);
            kid[h] = child ? sh.token[i] : -1;
            kx[h] = -INFINITY;
            ku[h] = 0.0f;
            kq[h] = 1.0f;
            if (kid[h] >= 0 && kid[h] < a.vocab) {
                kx[h] = logit<BF16>(row, kid[h]);
                ku[h] = a.u_accept[row0 + i];
                if (drafter) kq[h] = q[kid[h]];
            }
        }
        if (line >> cur & 1) {
            m = sh.node_top[cur];
            at = sh.node_best[cur];
        } else {
            if constexpr (KEEP) {
#pragma unroll
                for (int k = 0; k < kRegs; ++k)
                    if (v0 + k * kStep < v1) look(x[k], v0 + k * kStep + lane * kVec);
            } else {
                for (int64_t v = v0 + lane * kVec; v < v1; v += kAhead * kStep) {
                    float w[kAhead][kVec];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        if (v + k * kStep < v1) {
                            L::load(row, v + k * kStep, v1, w[k]);
                        } else {
#pragma unroll
                            for (int i = 0; i < kVec; ++i) w[k][i] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) look(w[k], v + k * kStep);
                }
            }
            warp_top(m, at);
            if (lane < C) {
                Shared* p = cl.map_shared_rank(&sh, lane);
                p->top[top_turn][me] = m;
                p->best[top_turn][me] = at;
            }
            cl.sync();
            m = -INFINITY;
            at = kNowhere;
            for (int i = lane; i < parts; i += 32)
                if (sh.top[top_turn][i] > m) {   // parts in order: the first place stays
                    m = sh.top[top_turn][i];
                    at = sh.best[top_turn][i];
                }
            warp_top(m, at);
            top_turn ^= 1;
        }
        const bool some = m > -INFINITY;   // else a row without weight
        const float top = fminf(m, FLT_MAX), rate = m == INFINITY ? 1.0f : rate_of;
        const int best = at;   // kNowhere: nothing above -inf
        int next = -1;
        if (greedy) {
            const unsigned b0 = __ballot_sync(0xffffffffu, kid[0] == best), b1 = __ballot_sync(0xffffffffu, kid[1] == best);
            if (length < a.path_stride && best != kNowhere) next = b0 ? __ffs(b0) - 1 : b1 ? 31 + __ffs(b1) : -1;
            if (next < 0) {
                if (rank == 0 && tid == 0) {
                    tokens[length - 1] = best == kNowhere ? -1 : best;
                    a.n_path[r] = length;
                }
                break;
            }
        } else {
            // What is likely to be read next: the first child's row, or, where the pieces have left the child open, the
            // drafter's row for what its refusal leaves.
            if (kids[0] | kids[1]) {
                const bool open = drafter && (line >> cur & 1);
                const int64_t c = kids[0] ? __ffs(kids[0]) - 1 : 31 + __ffs(kids[1]), es = open ? 4 : BF16 ? 2 : 4;
                const uint8_t* ahead = open ? reinterpret_cast<const uint8_t*>(q)
                                            : static_cast<const uint8_t*>(a.logits) + (row0 + c) * a.row_stride * es;
                for (int64_t b = v0 * es + lane * 128; b < v1 * es; b += 32 * 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(ahead + b));
            }
            // The row's sum; kept logits turn into weights.
            {
                Sum s;
                if constexpr (KEEP) {
#pragma unroll
                    for (int k = 0; k < kRegs; ++k)
                        if (v0 + k * kStep < v1 && some) {
                            weigh(x[k], top, rate);
                            s.add(x[k], fix);
                        }
                } else if (some) {
                    for (int64_t v = v0 + lane * kVec; v < v1; v += kAhead * kStep) {
                        s.room(fix);
                        float w[kAhead][kVec];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            if (v + k * kStep < v1) {
                                L::load(row, v + k * kStep, v1, w[k]);
                            } else {
#pragma unroll
                                for (int i = 0; i < kVec; ++i) w[k][i] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            weigh(w[k], top, rate);
                            s.add(w[k], fix);
                        }
                    }
                }
                exchange(warp_sum(s.value(fix)));
            }
            const int plain_turn = sum_turn;
            // The children, in order: the first warp of every CTA decides, all alike.
            float kw[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) kw[h] = kid[h] >= 0 && some ? weight(kx[h], top, rate) : 0.0f;
            unsigned todo[2] = {kids[0], kids[1]};
            uint64_t refused = 0;
            double tau = 0.0;
            for (;;) {
                const bool first = tau == 0.0;   // (before the first warp adds to it)
                if (warp == 0) {
                    int64_t total = total_of();
                    int got = -1;
                    bool again = false;   // a refusal that changes W everywhere
                    while (length < a.path_stride && (todo[0] | todo[1]) && !again) {
                        const int h = todo[0] ? 0 : 1, c = __ffs(todo[h]) - 1;
                        if (h) todo[1] &= todo[1] - 1;
                        else todo[0] &= todo[0] - 1;
                        const int y = __shfl_sync(0xffffffffu, h ? kid[1] : kid[0], c);
                        float w = __shfl_sync(0xffffffffu, h ? kw[1] : kw[0], c);
                        const float qy = __shfl_sync(0xffffffffu, h ? kq[1] : kq[0], c), u = __shfl_sync(0xffffffffu, h ? ku[1] : ku[0], c);
                        if (drafter) {
                            if (tau > 0.0) w = rest(w, (float)tau, qy);
                        } else {   // the same token on a child refused before
                            const bool gone = ((refused >> lane & 1) && kid[0] == y) || ((refused >> (lane + 32) & 1) && kid[1] == y);
                            if (__any_sync(0xffffffffu, gone)) w = 0.0f;
                        }
                        if ((double)u * (double)qy * ((double)total * fix.down) < (double)w) {
                            got = c + 32 * h;
                            break;
                        }
                        if (drafter) {
                            again = true;
                            tau += (double)total * fix.down;
                        } else if (w > 0.0f) {
                            refused |= 1ull << (c + 32 * h);
                            total = max(total - fix.of(w), (int64_t)0);
                        }
                    }
                    if (lane == 0) {
                        sh.next = got;
                        sh.again = again;
                        sh.tau = tau;
                        sh.refused = refused;
                    }
                }
                __syncthreads();
                next = sh.next;
                tau = sh.tau;
                if (!sh.again) break;
                if (first)   // the sums of e, for a row in which nothing will be left
                    for (int i = tid; i < parts; i += kThreads) sh.plain[i] = sh.sums[plain_turn][i];
                const float off = (float)tau;
                Sum s;
                if constexpr (KEEP) {
#pragma unroll
                    for (int k = 0; k < kRegs; ++k) {
                        const int64_t v = v0 + k * kStep + lane * kVec;
                        if (v < v1 && some) {
                            float q1[kVec];
                            load_q(v, q1);
#pragma unroll
                            for (int i = 0; i < kVec; ++i) q1[i] = rest(x[k][i], off, q1[i]);
                            s.add(q1, fix);
                        }
                    }
                } else if (some) {
                    constexpr int kTwo = kVec == 8 ? 1 : kVec == 4 ? 2 : 4;
                    for (int64_t v = v0 + lane * kVec; v < v1; v += kTwo * kStep) {
                        s.room(fix);
                        float w2[kTwo][kVec], q2[kTwo][kVec];
#pragma unroll
                        for (int k = 0; k < kTwo; ++k)
                            if (v + k * kStep < v1) {
                                L::load(row, v + k * kStep, v1, w2[k]);
                                load_q(v + k * kStep, q2[k]);
                            }
#pragma unroll
                        for (int k = 0; k < kTwo; ++k)
                            if (v + k * kStep < v1) {
                                weigh(w2[k], top, rate);
#pragma unroll
                                for (int i = 0; i < kVec; ++i) w2[k][i] = rest(w2[k][i], off, q2[k][i]);
                                s.add(w2[k], fix);
                            }
                    }
                }
                exchange(warp_sum(s.value(fix)));   // (and all have read the decision)
            }
        }
        if (next >= 0) {
            if (rank == 0 && tid == 0) {
                tokens[length - 1] = sh.token[next];
                path[length] = next;
            }
            cur = next;
            ++length;
            continue;
        }
        // The token after the path.  First the part that holds the threshold.
        __syncthreads();   // the decision has been read, sh.plain is written
        const uint64_t refused = sh.refused;
        const double tau = sh.tau;
        if (warp == 0) {
            if (refused)
                for (int i = lane; i < parts; i += 32) sh.plain[i] = sh.sums[sum_turn][i];
            __syncwarp();
            if (lane == 0)
                for (uint64_t left = refused; left; left &= left - 1) {   // tokens taken out of their parts' sums
                    const int y = sh.token[__ffsll((long long)left) - 1];
                    sh.sums[sum_turn][y / share] = max(sh.sums[sum_turn][y / share] - fix.of(weight(logit<BF16>(row, y), top, rate)), (int64_t)0);
                }
            __syncwarp();
            const bool usual = (tau == 0.0 && !refused) || total_of() > 0;   // else nothing is left: the row's own weights
            const int64_t* part = usual ? sh.sums[sum_turn] : sh.plain;
            const int each = (parts + 31) / 32;
            int64_t mine = 0;
            for (int k = 0; k < each; ++k)
                if (lane * each + k < parts) mine += part[lane * each + k];
            const int64_t upto = warp_scan(mine, lane), S = __shfl_sync(0xffffffffu, upto, 31);
            // sums above u S: above its whole part (u outside 0 .. 1 or NaN: some token all the same)
            const int64_t target = (int64_t)fmin(fmax((double)u_sample * (double)S, 0.0), 0x1p62);
            int64_t run = upto - mine, before = 0;
            int hit = kNowhere, last = -1;
            for (int k = 0; k < each; ++k) {
                const int i = lane * each + k;
                if (i < parts && part[i] > 0) {
                    last = i;
                    if (hit == kNowhere && run + part[i] > target) {
                        hit = i;
                        before = run;
                    }
                    run += part[i];
                }
            }
            const int found = __reduce_min_sync(0xffffffffu, hit);
            last = __reduce_max_sync(0xffffffffu, last);
            if (lane == 0) {
                sh.part = found != kNowhere ? found : last;   // none when the threshold is the end: the last token
                sh.target = found != kNowhere ? target : INT64_MAX;
                sh.before = 0;
                sh.usual = usual;
            }
            __syncwarp();
            if (found != kNowhere && hit == found) sh.before = before;
        }
        __syncthreads();
        const int part = sh.part;
        if (part < 0) {   // a row without weight
            if (rank == 0 && tid == 0) a.n_path[r] = length;
            break;
        }
        if (part / kWarps != rank) break;
        // Then the token: the part's CTA cuts it into pieces of whole steps, a warp each, in order.
        const bool usual = sh.usual != 0;
        const int64_t target = sh.target;
        const float off = usual ? (float)tau : 0.0f;
        const int64_t p0 = min((int64_t)part * share, a.vocab), p1 = min(p0 + share, a.vocab);
        const int64_t each = ((share / kStep + kWarps - 1) / kWarps) * kStep;
        const int64_t w0 = min(p0 + warp * each, p1), w1 = min(w0 + each, p1);
        auto weights = [&](int64_t v, float (&w)[kVec]) {   // W of kVec tokens from v on
            if (v >= w1) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) w[i] = 0.0f;
                return;
            }
            L::load(row, v, w1, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                w[i] = weight(w[i], top, rate);
                if (off > 0.0f && v + i < w1) w[i] = rest(w[i], off, q[v + i]);
            }
            for (uint64_t left = usual ? refused : 0; left; left &= left - 1) {
                const int y = sh.token[__ffsll((long long)left) - 1];
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (v + i == y) w[i] = 0.0f;
            }
        };
        int64_t mine = 0;
        for (int64_t b = w0; b < w1; b += kStep) {
            float w[kVec];
            weights(b + lane * kVec, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) mine += fix.of(w[i]);
        }
        mine = warp_sum(mine);
        if (lane == 0) sh.piece[warp] = mine;
        __syncthreads();
        int64_t run = sh.before;
        int mine_is = -1, last_is = -1;   // the warp whose piece holds the threshold; the last with weight
        for (int k = 0; k < kWarps; ++k) {
            const int64_t p = sh.piece[k];
            if (p > 0) {
                last_is = k;
                if (mine_is < 0) {
                    if (run + p > target) mine_is = k;
                    else run += p;
                }
            }
        }
        if (warp == (mine_is >= 0 ? mine_is : last_is < 0 ? 0 : last_is)) {
            const int64_t goal = mine_is >= 0 ? target : INT64_MAX;
            int token = -1, last = -1;
            for (int64_t b = w0; b < w1 && token < 0; b += kStep) {
                float w[kVec];
                weights(b + lane * kVec, w);
                int64_t sum = 0;
#pragma unroll
                for (int i = 0; i < kVec; ++i) sum += fix.of(w[i]);
                const int64_t upto = warp_scan(sum, lane);
                int64_t sofar = run + (upto - sum);
                int hit = kNowhere, some = -1;
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (w[i] > 0.0f) {
                        sofar += fix.of(w[i]);
                        some = (int)(b + lane * kVec + i);
                        if (hit == kNowhere && sofar > goal) hit = some;
                    }
                hit = __reduce_min_sync(0xffffffffu, hit);
                last = max(last, __reduce_max_sync(0xffffffffu, some));
                if (hit != kNowhere) token = hit;
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

template <bool BF16, bool VEC, bool KEEP>
static cudaError_t go(const VerifyArgs& a, int cluster, int per_row, int sms, cudaStream_t s) {
    Piece* pieces = per_row ? static_cast<Piece*>(a.ws) : nullptr;
    if (per_row) {
        // as many CTAs a request as its rows need, if it has its share of them, and no more than the GPU holds at once
        const int64_t rows = (a.n_rows + a.n_req - 1) / a.n_req;
        const int share = (int)std::max<int64_t>(1, std::min((std::min<int64_t>(rows, kNodes) * per_row + kPieceWarps - 1) / kPieceWarps,
                                                             kPieceCtas * sms / a.n_req));
        piece_kernel<BF16, VEC><<<(unsigned)(a.n_req * share), kPieceWarps * 32, 0, s>>>(a, pieces, per_row, share);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.n_req * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = per_row ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<BF16, VEC, KEEP>, a, (const Piece*)pieces, per_row);
}

template <bool BF16, bool VEC>
static cudaError_t go(const VerifyArgs& a, int cluster, int per_row, int sms, cudaStream_t s) {
    using L = vt::Lanes<BF16, VEC>;
    const int64_t parts = (int64_t)cluster * kWarps, share = ((a.vocab + parts - 1) / parts + L::kStep - 1) / L::kStep;
    return share * L::kVec <= kKeep ? go<BF16, VEC, true>(a, cluster, per_row, sms, s) : go<BF16, VEC, false>(a, cluster, per_row, sms, s);
}

}  // namespace vt

// Pieces of a row that are summed first, or 0: where no request can have a
// child, where a row has too many tokens for their margin, and where they would
// take more than 256 MiB.
static int pieces_of(int64_t n_rows, int64_t n_req, int64_t vocab) {
    const int64_t per_row = (vocab + vt::kPiece - 1) / vt::kPiece;
    return n_rows <= n_req || vocab > vt::kPieceVocab || n_rows * per_row > 1 << 24 ? 0 : (int)per_row;
}

int64_t verify_ws_bytes(int64_t n_rows, int64_t n_req, int64_t vocab) {
    return n_rows * pieces_of(n_rows, n_req, vocab) * (int64_t)sizeof(vt::Piece);
}

cudaError_t launch_verify_tree(const VerifyArgs& a, int sms, cudaStream_t s) {
    // CTAs of a request: as many as leave each some thousand tokens and all of them a place at once.
    const int cluster = (int)std::max<int64_t>(1, std::min<int64_t>({vt::kMaxCluster, 2 * sms / a.n_req, a.vocab / 1024}));
    const int es = a.bf16 ? 2 : 4;
    const bool vec = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.row_stride * es % 16 == 0;
    VerifyArgs b = a;
    b.probs_vec = reinterpret_cast<uintptr_t>(a.probs) % 16 == 0 && a.probs_stride % 4 == 0;
    const int per_row = pieces_of(a.n_rows, a.n_req, a.vocab);
    if (a.bf16) return vec ? vt::go<true, true>(b, cluster, per_row, sms, s) : vt::go<true, false>(b, cluster, per_row, sms, s);
    return vec ? vt::go<false, true>(b, cluster, per_row, sms, s) : vt::go<false, false>(b, cluster, per_row, sms, s);
}

}  // namespace qk
