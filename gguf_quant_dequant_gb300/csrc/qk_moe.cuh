// qk_moe.cuh -- the products of a mixture-of-experts layer over packed expert
// weights for a few tokens (qk_moe_ffn): h = SiLU(Wg x) * (Wu x) of every
// (token, expert) pair, then the gate-weighted sum of Wd h over a token's
// experts.
//
// A decode batch meets few tokens per expert, so the weights of the experts
// met are streamed once and the work per weight is that of the decode GEMV
// (qk_hgemv.cu): 16-row tiles in a ring of shared-memory stages filled by bulk
// copies, one warp per 256-weight unit, exact codes on the fp16 warp MMA
// against activations as two fp16 terms (qk_hunits.cuh).  What differs:
//   * pairs are grouped by expert (at most kGroup to a group) in every CTA, from
//     the ids alone; a stage's weights serve all pairs of the group, two at a
//     time;
//   * up: groups x rows, weighted by their pairs, are cut into one contiguous
//     range per CTA; the SiLU and the product are the end of a tile;
//   * down: a CTA has 16 rows of the output and walks all groups, so that the
//     sum over experts stays in its shared memory, in the groups' order;
//   * short rows (fewer than eight units) put several tiles into a stage, so that
//     all eight warps have one;
//   * each warp leaves its partial sums beside the stage; the warp that refills
//     the stage adds them up in warp order first.  No barrier joins the
//     consumers after the start, and the result does not depend on timing.
#pragma once
#include <algorithm>
#include <cooperative_groups.h>
#include <type_traits>

#include "qk_formats.cuh"
#include "qk_hunits.cuh"
#include "qk_hx.cuh"
#include "qk_internal.h"
#include "qk_ptx.cuh"

namespace cg = cooperative_groups;

namespace qk {
namespace moe {
using namespace hm;

constexpr int kCW = 8;                      // consumer warps
constexpr int kThreads = (kCW + 1) * 32;    // + the warp that fills stages and adds up
constexpr int kTileRows = 16;
constexpr int kUnitW = 256;
constexpr int kGroup = 8;                   // most pairs of a group
constexpr int kMaxStages = 8;
constexpr uint16_t kNone = 0xffff;

struct Args {
    const float* x;             // up: [n_tok, cols]; down: h [pairs, cols]
    int64_t cols, rows;         // of one expert's matrix
    uint32_t row_bytes;
    const uint8_t *W0, *W1;     // up: gate and up matrices; down: its matrix
    int n_exp, n_tok, k, pairs;
    const float* logits;        // router's logits [n_tok, n_exp] (up only), or nullptr: ids are given
    bool norm;
    float scale;
    int32_t* ids;               // [n_tok, k]
    float* gate;
    float* out;                 // up: h [pairs, rows]; down: [n_tok, rows]
    int nxb, nunits, nchunks;   // of a row: 32-blocks, units, chunks of eight units
    int nu, subs, stages;       // units and tiles of a stage; ring depth
    int gcap;                   // most pairs of a group in this call
    uint32_t slot, stage_bytes; // of a row; of a stage without its partial sums
    int entries;                // up, long rows: (tile, pair) sums kept between chunks
    int gmax, quantum;          // groups the tables hold; up: rows that stay together
    int split;                  // down: CTAs (a cluster) that share a tile of the output
    uint32_t off_xm, off_xs, off_acc, off_pairs, off_gexp, off_gbeg, off_gcnt, off_cost, off_gate, off_bar, off_part, off_ring;
    unsigned* status;
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// ------------------------------------------------------- choice of experts --
// Order-preserving image of a float: one for both zeros, NaN above all.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v), mag = u & 0x7fffffffu;
    if (mag > 0x7f800000u) return 0xffffffffu;
    return (u >> 31) && mag ? ~u : mag | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

// One warp, one token: the k largest of n logits (the lowest index of equals),
// their softmax over all n or over the k.
template <int NE>
__device__ __forceinline__ void choose(const float* lg, int n, int k, bool norm, float scale, int lane, uint16_t* ids, int32_t* ids_out,
                                       float* gate_out) {
    uint32_t key[NE];
    float l[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < n ? __ldcg(lg + e) : -INFINITY;
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
        if (lane == 0) {
            ids[j] = (uint16_t)at;
            if (ids_out) ids_out[j] = at;
        }
    }
    if (!norm) {
#pragma unroll
        for (int i = 0; i < NE; ++i) sum += lane + 32 * i < n ? expf(l[i] - top) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (gate_out && lane < k) gate_out[lane] = mine / sum * scale;
}

// Shared-memory tables of the groups.
struct Tables {
    uint16_t *pairs, *gexp, *gbeg, *gcnt;   // pairs by expert; expert, first pair and pairs of a group
    uint32_t* cost;                         // up: running cost of the groups' quanta
    float* gate;                            // down
    int* n;                                 // number of groups
};

// Work of a row tile by its pairs, in twentieths of a single token's: two at
// a time share the conversion of the codes.
__device__ __forceinline__ uint32_t cost_of(int n) { return (uint32_t)(28 * (n >> 1) + 20 * (n & 1)); }

// ids (shared, one per pair, kNone = none) -> groups.  scratch: 2 * n_exp
// words of shared memory.
__device__ inline void build_groups(const Args& p, const Tables& t, const uint16_t* ids, int* scratch) {
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t quanta = (uint32_t)((p.rows + p.quantum - 1) / p.quantum);
    if (p.n_tok == 1 || p.gcap == 1) {   // every pair is a group of its own
        if (tid < 32) {
            int n = 0;
            uint32_t cost = 0;
            for (int b = 0; b < p.pairs; b += 32) {
                const bool ok = b + lane < p.pairs && ids[b + lane] != kNone;
                const unsigned m = __ballot_sync(0xffffffffu, ok);
                const int at = n + __popc(m & ((1u << lane) - 1));
                if (ok) {
                    t.pairs[at] = (uint16_t)(b + lane);
                    t.gexp[at] = ids[b + lane];
                    t.gbeg[at] = (uint16_t)at;
                    t.gcnt[at] = 1;
                    if (t.cost) t.cost[at] = (uint32_t)at * cost_of(1) * quanta;
                }
                n += __popc(m);
            }
            cost = (uint32_t)n * cost_of(1) * quanta;
            if (lane == 0) {
                if (t.cost) t.cost[n] = cost;
                *t.n = n;
            }
        }
        return;
    }
    int* count = scratch;
    int* offs = scratch + p.n_exp;
    for (int e = tid; e < p.n_exp; e += kThreads) count[e] = 0;
    __syncthreads();
    for (int i = tid; i < p.pairs; i += kThreads)
        if (ids[i] != kNone) atomicAdd(&count[ids[i]], 1);
    __syncthreads();
    if (tid >= 32) return;
    // Experts in order, a run of them per lane: running sums of pairs, groups and cost.
    const int per = (p.n_exp + 31) / 32, e0 = lane * per, e1 = min(e0 + per, p.n_exp);
    int np = 0, ng = 0;
    uint32_t cs = 0;
    for (int e = e0; e < e1; ++e) {
        const int c = count[e];
        np += c;
        ng += (c + p.gcap - 1) / p.gcap;
        cs += (uint32_t)(c / p.gcap) * cost_of(p.gcap) + cost_of(c % p.gcap);
    }
    int ip = np, ig = ng;
    uint32_t ic = cs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, ip, o), b = __shfl_up_sync(0xffffffffu, ig, o);
        const uint32_t c = __shfl_up_sync(0xffffffffu, ic, o);
        if (lane >= o) {
            ip += a;
            ig += b;
            ic += c;
        }
    }
    if (lane == 31) {
        *t.n = ig;
        if (t.cost) t.cost[ig] = ic * quanta;
    }
    ip -= np;
    ig -= ng;
    ic -= cs;
    for (int e = e0; e < e1; ++e) {
        offs[e] = ip;
        for (int c = count[e]; c > 0; c -= p.gcap) {
            const int m = min(c, p.gcap);
            t.gexp[ig] = (uint16_t)e;
            t.gbeg[ig] = (uint16_t)ip;
            t.gcnt[ig] = (uint16_t)m;
            if (t.cost) t.cost[ig] = ic * quanta;
            ic += cost_of(m);
            ip += m;
            ++ig;
        }
    }
    __syncwarp();
    // Pairs into their expert's run, in order.
    for (int b = 0; b < p.pairs; b += 32) {
        const int i = b + lane;
        const int e = i < p.pairs ? ids[i] : kNone;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int at = 0;
        if (e != kNone) {
            at = offs[e] + __popc(same & ((1u << lane) - 1));
            t.pairs[at] = (uint16_t)i;
        }
        __syncwarp();
        if (e != kNone && lane == 31 - __clz((int)same)) offs[e] = at + 1;
        __syncwarp();
    }
}

// ------------------------------------------------------------- the order --
// The stages of a CTA, in the order in which they are filled and used; every
// warp walks its own copy.
// up: the CTA's groups; of each its rows in batches of tiles; of each batch the
// chunks of K; of each chunk the (tile, gate or up) items, `subs` to a stage.
struct UpIter {
    int g, ng, c, i, ni, t0, nt, tiles, r0, r1;
    int64_t lo, hi;   // the CTA's share of the cost, times the grid
    __device__ __forceinline__ void start(const Args& p, const Tables& t) {
        ng = *t.n;
        const int64_t total = t.cost[ng];
        lo = total * blockIdx.x;
        hi = total * (blockIdx.x + 1);
        // the last group that begins at or before the share
        int a = 0, b = ng;
        while (a < b) {
            const int m = (a + b + 1) >> 1;
            if (m < ng && (int64_t)t.cost[m] * gridDim.x <= lo) a = m;
            else b = m - 1;
        }
        g = a - 1;
        next_group(p, t);
    }
    __device__ __forceinline__ bool valid() const { return g < ng; }
    __device__ __forceinline__ void next_group(const Args& p, const Tables& t) {
        const int64_t G = gridDim.x, nq = (p.rows + p.quantum - 1) / p.quantum;
        for (++g; g < ng; ++g) {
            const int64_t base = (int64_t)t.cost[g] * G, w = (int64_t)cost_of(t.gcnt[g]) * G;
            if (base >= hi) {
                g = ng;
                break;
            }
            // quantum q belongs to the CTA whose share holds base + q w
            const int64_t q0 = lo > base ? (lo - base + w - 1) / w : 0, q1 = min(nq, (hi - base + w - 1) / w);
            if (q0 < q1) {
                r0 = (int)(q0 * p.quantum);
                r1 = (int)min(q1 * p.quantum, p.rows);
                tiles = (r1 - r0 + kTileRows - 1) / kTileRows;
                c = 0;
                batch(p, t, 0);
                return;
            }
        }
    }
    __device__ __forceinline__ void batch(const Args& p, const Tables& t, int from) {
        t0 = from;
        nt = tiles - from;
        if (p.nchunks > 1) nt = min(nt, max(1, p.entries / (int)t.gcnt[g]));
        ni = (2 * nt + p.subs - 1) / p.subs;
        i = 0;
    }
    // To the next chunk of activations: another chunk, batch or group.
    __device__ __forceinline__ void next_chunk(const Args& p, const Tables& t) {
        i = 0;
        if (++c < p.nchunks) return;
        c = 0;
        if (t0 + nt < tiles) batch(p, t, t0 + nt);
        else next_group(p, t);
    }
    __device__ __forceinline__ void next(const Args& p, const Tables& t) {
        if (++i >= ni) next_chunk(p, t);
    }
    // The item of tile slot `sub`: its group, or -1.
    __device__ __forceinline__ int group(const Args& p, int sub) const { return i * p.subs + sub < 2 * nt ? g : -1; }
};
// down: the groups, `subs` to a stage (chunks of a long row one after another).
// The CTAs that share a tile take every split-th stage.
struct DownIter {
    int i, c, ng;
    __device__ __forceinline__ void start(const Args& p, const Tables& t) {
        i = c = 0;
        ng = *t.n;
        for (int k = blockIdx.x % (unsigned)p.split; k > 0; --k) step(p);
    }
    __device__ __forceinline__ bool valid() const { return i < ng; }
    __device__ __forceinline__ void step(const Args& p) {
        if (++c == p.nchunks) {
            c = 0;
            i += p.subs;
        }
    }
    __device__ __forceinline__ void next(const Args& p, const Tables&) {
        for (int k = 0; k < p.split; ++k) step(p);
    }
    __device__ __forceinline__ void next_chunk(const Args& p, const Tables& t) { next(p, t); }
    __device__ __forceinline__ int group(const Args&, int sub) const { return i + sub < ng ? i + sub : -1; }
};

// ----------------------------------------------------------------- kernel --
// MT: pairs per pass over a stage's codes (1 when every group has one pair).
template <int T, int MT, bool DOWN>
__global__ void __launch_bounds__(kThreads, 2) moe_kernel(const Args p) {
    using U = HU<T>;
    using Iter = typename std::conditional<DOWN, DownIter, UpIter>::type;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);
    uint64_t* empty = full + kMaxStages;
    volatile int* abort = reinterpret_cast<volatile int*>(empty + kMaxStages);
    Tables tb;
    tb.pairs = reinterpret_cast<uint16_t*>(smem + p.off_pairs);
    tb.gexp = reinterpret_cast<uint16_t*>(smem + p.off_gexp);
    tb.gbeg = reinterpret_cast<uint16_t*>(smem + p.off_gbeg);
    tb.gcnt = reinterpret_cast<uint16_t*>(smem + p.off_gcnt);
    tb.cost = DOWN ? nullptr : reinterpret_cast<uint32_t*>(smem + p.off_cost);
    tb.gate = DOWN ? reinterpret_cast<float*>(smem + p.off_gate) : nullptr;
    tb.n = const_cast<int*>(reinterpret_cast<volatile int*>(empty + kMaxStages)) + 1;
    float* acc = reinterpret_cast<float*>(smem + p.off_acc);
    float* part = reinterpret_cast<float*>(smem + p.off_part);   // [stage][warp][gcap][16]
    uint8_t* ring = smem + p.off_ring;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rb = p.row_bytes;
    const int part_stage = kCW * p.gcap * kTileRows;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kCW);
        }
        *abort = 0;
        fence_barrier_init();
    }
    pdl_launch_dependents();
    pdl_wait_prior();   // the router's logits, or h, the ids and the gates
    {
        uint16_t* ids = reinterpret_cast<uint16_t*>(ring);   // before the first stage
        int* scratch = reinterpret_cast<int*>(ring + 2 * ((p.pairs + 7) & ~7));
        if (!DOWN && p.logits) {
            for (int tok = warp; tok < p.n_tok; tok += kCW + 1) {
                const float* lg = p.logits + (int64_t)tok * p.n_exp;
                int32_t* io = blockIdx.x == 0 ? p.ids + (int64_t)tok * p.k : nullptr;
                float* go = blockIdx.x == 0 ? p.gate + (int64_t)tok * p.k : nullptr;
                if (p.n_exp <= 128) choose<4>(lg, p.n_exp, p.k, p.norm, p.scale, lane, ids + tok * p.k, io, go);
                else if (p.n_exp <= 256) choose<8>(lg, p.n_exp, p.k, p.norm, p.scale, lane, ids + tok * p.k, io, go);
                else choose<16>(lg, p.n_exp, p.k, p.norm, p.scale, lane, ids + tok * p.k, io, go);
            }
        } else {
            for (int i = threadIdx.x; i < p.pairs; i += kThreads) {
                const int e = __ldcg(p.ids + i);
                ids[i] = e >= 0 && e < p.n_exp ? (uint16_t)e : kNone;
                if (DOWN) tb.gate[i] = __ldcg(p.gate + i);
            }
        }
        __syncthreads();
        build_groups(p, tb, ids, scratch);
        fence_proxy_async_smem();   // the ring's first copies come after these uses of it
        __syncthreads();
    }
    // down: this CTA's rows of the output.
    const int64_t dtiles = DOWN ? gridDim.x / p.split : 1, dt = DOWN ? blockIdx.x / p.split : 0;
    const int64_t rq = p.rows / dtiles, rr = p.rows % dtiles;
    const int64_t d0 = DOWN ? dt * rq + min(dt, rr) : 0;
    const int drows = DOWN ? (int)(rq + (dt < rr ? 1 : 0)) : 0;

    // ---------------- consumers ----------------
    auto consume = [&]() {
        const int g8 = lane >> 2, t = lane & 3;
        uint8_t* xbw = smem + warp * MT * (8 * kXBB);
        float4* xmw = reinterpret_cast<float4*>(smem + p.off_xm) + warp * MT * 8;
        float* xsw = reinterpret_cast<float*>(smem + p.off_xs) + warp * MT * kUnitW;
        const bool owner = (g8 >> 1) == t;
        const int sub = warp / p.nu, uic = warp - sub * p.nu;
        float* mypart = part + warp * p.gcap * kTileRows;
        // A step of a warp: one stage, and MT pairs of its group; it needs their activations of the warp's unit.
        auto group_of = [&](const Iter& d) -> int {
            if (sub >= p.subs || !d.valid() || d.c * kCW + uic >= p.nunits) return -1;
            return d.group(p, sub);
        };
        auto stage_x = [&](const Iter& d, int g, int sg) {   // asks for the activations of a step
            const int n = tb.gcnt[g], beg = tb.gbeg[g], u = d.c * kCW + uic;
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (sg * MT + m < n) {
                    const int pair = tb.pairs[beg + sg * MT + m];
                    load_unit_x(p.x + (int64_t)(DOWN ? pair : pair / p.k) * p.cols, p.nxb, u, lane, xsw + m * kUnitW);
                }
            cp_async_commit();
        };
        Iter it, ahead;
        it.start(p, tb);
        // `ahead` is the stage whose first step's activations are asked for next.
        ahead = it;
        auto seek = [&]() {   // to the next stage in which this warp has work
            while (ahead.valid() && group_of(ahead) < 0) ahead.next(p, tb);
        };
        seek();
        if (ahead.valid()) stage_x(ahead, group_of(ahead), 0);
        int s = 0;
        uint32_t ph = 0;
        bool dead = false;
        using BP1 = typename std::conditional<MT == 1, BRegs, BSmem<1>>::type;
        BP1 b1 = {};
        const uint32_t xo0 = (U::X0(t) * 2 + (g8 & 1)) * 64, xo1 = (U::X1(t) * 2 + (g8 & 1)) * 64;
        for (; it.valid(); it.next(p, tb)) {
            const int g = group_of(it);
            bool waited = false;
            if (g >= 0) {
                const int n = tb.gcnt[g], u = it.c * kCW + uic, nvb = min(8, p.nxb - 8 * u);
                // Rows g8 and g8 + 8 start (row * row_bytes) mod 16 bytes into their slots (a chunk is a multiple of 16 bytes).
                int64_t row;
                if constexpr (DOWN) row = (int64_t)tb.gexp[g] * p.rows + d0 + g8;
                else row = (int64_t)tb.gexp[g] * p.rows + it.r0 + (int64_t)(it.t0 + ((it.i * p.subs + sub) >> 1)) * kTileRows + g8;
                const uint8_t* q0 = ring + (uint32_t)s * p.stage_bytes + (sub * kTileRows + g8) * p.slot + uic * U::UB;
                const uint8_t* q1 = q0 + 8 * p.slot + (((uint32_t)(row + 8) * rb) & 15u);
                q0 += ((uint32_t)row * rb) & 15u;
                const int nsg = (n + MT - 1) / MT;
                // up: one group's tiles of a chunk share their activations (a warp with work in any has it in the first)
                bool first = true;
                if constexpr (!DOWN) first = it.i == 0;
                for (int sg = 0; sg < nsg; ++sg) {
                    const int live = min(MT, n - sg * MT);
                    if (DOWN || nsg > 1 || first) {
                        cp_async_wait<0>();
                        __syncwarp();   // every lane is done with the activations before
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            if (m < live) prep_unit_x(xsw + m * kUnitW, xbw + m * (8 * kXBB), xmw + m * 8, lane);
                        __syncwarp();
                        if (sg + 1 < nsg) {
                            stage_x(it, g, sg + 1);
                        } else {
                            // the next step that needs activations of its own
                            ahead = it;
                            if (!DOWN && nsg == 1) ahead.next_chunk(p, tb);
                            else ahead.next(p, tb);
                            seek();
                            if (ahead.valid()) stage_x(ahead, group_of(ahead), 0);
                        }
                        if constexpr (MT == 1) {
                            if (owner) {
                                load_xb(xbw + xo0, b1.x0);
                                load_xb(xbw + xo1, b1.x1);
                            }
                        }
                    }
                    if (!waited) {
                        waited = true;
                        if (!dead && !mbar_wait_abortable(&full[s], ph, p.status, abort)) dead = true;
                    }
                    float y0[MT], y1[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) y0[m] = y1[m] = 0.0f;
                    if (!dead) {
                        float4 xm0[MT], xm1[MT];
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            xm0[m] = xmw[m * 8 + U::X0(t)];
                            xm1[m] = xmw[m * 8 + U::X1(t)];
                        }
                        if constexpr (MT == 1) {
                            run_unit<T, 1>(q0, q1, b1, xm0, xm1, t, nvb, y0, y1);
                        } else {
                            if (live == 1) {
                                b1.own = owner;
                                b1.p[0][0] = xbw + xo0;
                                b1.p[0][1] = xbw + xo1;
                                float z0[1] = {0.0f}, z1[1] = {0.0f};
                                const float4 m0[1] = {xm0[0]}, m1[1] = {xm1[0]};
                                run_unit<T, 1>(q0, q1, b1, m0, m1, t, nvb, z0, z1);
                                y0[0] = z0[0];
                                y1[0] = z1[0];
                            } else {
                                BSmem<MT> bp;
                                bp.own = owner;
#pragma unroll
                                for (int m = 0; m < MT; ++m) {
                                    bp.p[m][0] = xbw + m * (8 * kXBB) + xo0;
                                    bp.p[m][1] = xbw + m * (8 * kXBB) + xo1;
                                }
                                run_unit<T, MT>(q0, q1, bp, xm0, xm1, t, nvb, y0, y1);
                            }
                        }
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        y0[m] += __shfl_xor_sync(0xffffffffu, y0[m], 1);
                        y1[m] += __shfl_xor_sync(0xffffffffu, y1[m], 1);
                        y0[m] += __shfl_xor_sync(0xffffffffu, y0[m], 2);
                        y1[m] += __shfl_xor_sync(0xffffffffu, y1[m], 2);
                        if (t < 2 && m < live) mypart[s * part_stage + (sg * MT + m) * kTileRows + t * 8 + g8] = t ? y1[m] : y0[m];
                    }
                }
            }
            if (!waited && !dead && !mbar_wait_abortable(&full[s], ph, p.status, abort)) dead = true;
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        cp_async_wait<0>();
    };

    if (warp == kCW) {
        // ---------------- fills stages, adds up the consumers' sums ----------------
        if (DOWN) {
            for (int i = lane; i < p.n_tok * kTileRows; i += 32) acc[i] = 0.0f;
            __syncwarp();
        }
        const uint64_t pol = policy_evict_first();
        const int64_t total16 = (p.n_exp * p.rows * (int64_t)rb) & ~(int64_t)15;
        // The sums of a used stage: row lane % 16, the warps of even or odd index by the half warp.
        auto add_up = [&](const Iter& d, int s) {
            const int row = lane & 15, half = lane >> 4;
            const int nw = min(p.nu, p.nunits - d.c * kCW);
            for (int sub = 0; sub < p.subs; ++sub) {
                const int g = d.group(p, sub);
                if (g < 0) break;
                const int n = tb.gcnt[g], beg = tb.gbeg[g];
                for (int j = 0; j < n; ++j) {
                    const float* q = part + s * part_stage + (sub * p.nu * p.gcap + j) * kTileRows + row;
                    float v = 0.0f;
                    for (int w = half; w < nw; w += 2) v += q[w * p.gcap * kTileRows];
                    v += __shfl_xor_sync(0xffffffffu, v, 16);
                    const int pair = tb.pairs[beg + j];
                    if constexpr (DOWN) {
                        if (half == 0) acc[pair / p.k * kTileRows + row] += tb.gate[pair] * v;
                    } else {
                        const int item = d.i * p.subs + sub, tile = item >> 1, pass = item & 1;
                        float* a = acc + (((p.nchunks > 1 ? tile : 0) * n + j) * 2 + pass) * kTileRows + row;
                        if (half == 0) {
                            if (d.c > 0) v += *a;
                            if (pass == 0 || d.c + 1 < p.nchunks) {
                                *a = v;
                            } else {
                                const float gv = a[-kTileRows];
                                const int r = d.r0 + (d.t0 + tile) * kTileRows + row;
                                if (r < d.r1) p.out[(int64_t)pair * p.rows + r] = gv / (1.0f + expf(-gv)) * v;
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        };
        Iter it, done;
        it.start(p, tb);
        done = it;
        int s = 0, filled = 0, added = 0;
        uint32_t ph = 0;
        bool dead = false;
        for (; it.valid() && !dead; it.next(p, tb)) {
            const bool again = filled >= p.stages;
            if (again && !mbar_wait_abortable(&empty[s], ph ^ 1u, p.status, abort)) {
                dead = true;
                break;
            }
            uint8_t* st = ring + (uint32_t)s * p.stage_bytes;
            const int64_t coff = (int64_t)it.c * kCW * U::UB;
            const int64_t len = min((int64_t)p.nu * U::UB, (int64_t)rb - coff);
            // Rows: tile slot q / 16, row q % 16.
            for (int q0 = 0; q0 < p.subs * kTileRows; q0 += 32) {
                const int q = q0 + lane, sub = q >> 4, row = q & 15;
                const int g = sub < p.subs ? it.group(p, sub) : -1;
                const uint8_t* W = p.W0;
                int64_t r = 0;
                bool live = g >= 0;
                if (live) {
                    if constexpr (DOWN) {
                        live = row < drows;
                        r = (int64_t)tb.gexp[g] * p.rows + d0 + row;
                    } else {
                        const int item = it.i * p.subs + sub;
                        const int rt = it.r0 + (it.t0 + (item >> 1)) * kTileRows + row;
                        live = rt < it.r1;
                        r = (int64_t)tb.gexp[g] * p.rows + rt;
                        if (item & 1) W = p.W1;
                    }
                }
                uint32_t bytes = 0;
                const int64_t off = r * rb + coff, a = off & ~(int64_t)15;
                if (live) {
                    const int64_t e = min((off + len + 15) & ~(int64_t)15, total16);
                    bytes = e > a ? (uint32_t)(e - a) : 0u;
                    // Bytes past the last full 16 bytes of the matrices.
                    for (int64_t b = max(off, total16); b < off + len; ++b) st[q * p.slot + (uint32_t)(b - a)] = W[b];
                }
                uint32_t total = bytes;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                if (lane == 0) mbar_expect_tx(&full[s], total);
                __syncwarp();
                if (bytes) bulk_g2s(st + q * p.slot, W + a, bytes, &full[s], pol);
            }
            if (again) {   // the sums that were left beside the stage, before its next users may write theirs
                add_up(done, s);
                done.next(p, tb);
                ++added;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
            ++filled;
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (!dead) {
            // The stages still in use, in their order.
            for (; added < filled; ++added) {
                const int t = added % p.stages;
                if (!mbar_wait_abortable(&empty[t], (uint32_t)(added / p.stages) & 1u, p.status, abort)) {
                    dead = true;
                    break;
                }
                add_up(done, t);
                done.next(p, tb);
            }
        }
        if (dead) {
            // Let the copies already requested land before the CTA exits.
            for (int k = max(0, filled - p.stages); k < filled; ++k)
                mbar_wait_bounded(&full[k % p.stages], (uint32_t)(k / p.stages) & 1u, p.status);
        } else if (DOWN && p.split == 1) {
            for (int i = lane; i < p.n_tok * kTileRows; i += 32) {
                const int row = i & 15;
                if (row < drows) p.out[(int64_t)(i >> 4) * p.rows + d0 + row] = acc[i];
            }
        }
    } else {
        consume();
    }

    if constexpr (DOWN) {
        if (p.split > 1) {
            // The sums of the tile's other CTAs, in their order.
            cg::cluster_group cl = cg::this_cluster();
            cl.sync();
            if (cl.block_rank() == 0) {
                for (int i = threadIdx.x; i < p.n_tok * kTileRows; i += kThreads) {
                    float v = acc[i];
                    for (int r = 1; r < p.split; ++r) v += cl.map_shared_rank(acc, r)[i];
                    const int row = i & 15;
                    if (row < drows) p.out[(int64_t)(i >> 4) * p.rows + d0 + row] = v;
                }
            }
            cl.sync();   // nobody leaves while its sums are read
        }
    }
}

// ------------------------------------------------------------------- host --
constexpr int64_t kSmemBudget = 113 * 1024;   // two CTAs per SM

inline int block_bytes(int type) {
    switch (type) {
    case T_Q4_K: return 144;
    case T_Q6_K: return 210;
    case T_Q8_0: return 34;
    case T_Q5_0: return 22;
    case T_Q4_0: return 18;
    case T_Q5_K: return 176;
    case T_Q2_K: return 84;
    case T_Q3_K: return 110;
    }
    return 0;
}
inline int block_elems(int type) { return type == T_Q8_0 || type == T_Q5_0 || type == T_Q4_0 ? 32 : 256; }

// Fills the geometry of one of the two products; returns its grid (0: none
// fits) and shared memory.
inline int plan(Args& a, int type, bool down, int sms, uint32_t* smem) {
    const int BB = block_bytes(type), BE = block_elems(type);
    a.row_bytes = (uint32_t)(a.cols / BE * BB);
    a.nxb = (int)(a.cols / 32);
    a.nunits = (int)((a.cols + kUnitW - 1) / kUnitW);
    a.nchunks = (a.nunits + kCW - 1) / kCW;
    a.nu = std::min(a.nunits, kCW);
    a.subs = kCW / a.nu;
    const int64_t UB = (int64_t)(kUnitW / BE) * BB, CB = a.nu * UB;
    // Room for the alignment remainder and word reads past the end, and a stride of 16 mod 32 bytes (banks).
    a.slot = (uint32_t)(((CB + 15 + 15) & ~(int64_t)15) + 16);
    if (a.slot % 32 == 0) a.slot += 16;
    a.stage_bytes = (uint32_t)a.subs * kTileRows * a.slot;
    const int mt = a.n_tok == 1 ? 1 : 2;
    // Two CTAs per SM; one where tables and stages leave no room for two.  Of the sizes of groups (larger ones read weights
    // less often) and of the sums kept between chunks (more tiles share their activations), the largest that leave three
    // stages, else the most stages.
    int best = 0;
    for (const int64_t budget : {kSmemBudget, 2 * kSmemBudget}) {
        Args chosen = a;
        for (int cap = a.n_tok == 1 ? 1 : kGroup; cap >= mt && best < 3; cap >>= 1)
            for (int entries = 64; entries >= cap && best < 3; entries >>= 1) {
                Args b = a;
                b.gcap = cap;
                b.entries = entries;
                b.gmax = a.n_tok == 1 ? a.pairs : std::min(a.pairs, a.n_exp + a.pairs / cap);
                int64_t at = (int64_t)kCW * mt * 8 * kXBB;
                auto take = [&](int64_t bytes) {
                    const int64_t o = at;
                    at = (at + bytes + 15) & ~(int64_t)15;
                    return (uint32_t)o;
                };
                b.off_xm = take((int64_t)kCW * mt * 8 * 16);
                b.off_xs = take((int64_t)kCW * mt * kUnitW * 4);
                b.off_acc = take(down ? (int64_t)a.n_tok * kTileRows * 4 : (int64_t)(a.nchunks > 1 ? entries : cap) * 2 * kTileRows * 4);
                b.off_pairs = take(2 * a.pairs);
                b.off_gexp = take(2 * b.gmax);
                b.off_gbeg = take(2 * b.gmax);
                b.off_gcnt = take(2 * b.gmax);
                b.off_cost = down ? 0 : take(4 * (b.gmax + 1));
                b.off_gate = down ? take(4 * a.pairs) : 0;
                b.off_bar = take(2 * kMaxStages * 8 + 16);
                const int64_t part = (int64_t)kCW * cap * kTileRows * 4;
                const int64_t n = std::min<int64_t>((budget - at - 128) / (a.stage_bytes + part), kMaxStages);
                // the ring also holds the ids and the counts while the groups are made
                if (n < 2 || n <= best || n * a.stage_bytes < 2 * ((a.pairs + 7) & ~7) + 8 * a.n_exp) continue;
                best = (int)n;
                b.stages = (int)n;
                b.off_part = take(n * part);
                b.off_ring = (uint32_t)((at + 127) & ~(int64_t)127);
                *smem = b.off_ring + (uint32_t)(n * a.stage_bytes);
                chosen = b;
            }
        if (best) {
            a = chosen;
            break;
        }
    }
    if (best == 0) return 0;
    const int64_t G = 2 * (int64_t)sms;
    if (down) {
        const int64_t tiles = (a.rows + kTileRows - 1) / kTileRows;
        a.split = 1;
        while (a.split < 8 && tiles * a.split * 2 <= G) a.split *= 2;
        // where every tile has a CTA, rows are dealt out evenly over as many as there is room for
        return (int)(a.split > 1 ? tiles * a.split : std::max(tiles, std::min(G, a.rows)));
    }
    a.split = 1;
    // experts that the pairs meet if they are spread evenly
    const double met = std::min<double>(a.n_exp, a.pairs);
    const double tiles = met * ((a.rows + kTileRows - 1) / kTileRows);
    a.quantum = tiles >= 3.0 * G ? kTileRows : 1;
    return (int)std::min<double>((double)G, met * a.rows);
}

template <int T, int MT, bool DOWN>
cudaError_t go(const Args& a, int grid, uint32_t smem, cudaStream_t s) {
    auto kern = moe_kernel<T, MT, DOWN>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(2 * kSmemBudget));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool DOWN>
cudaError_t launch_product(int type, Args& a, int sms, cudaStream_t s) {
    uint32_t smem = 0;
    const int grid = plan(a, type, DOWN, sms, &smem);
    if (grid == 0) return cudaErrorInvalidValue;
    const bool one = a.n_tok == 1;
    switch (type) {
    case T_Q4_K: return one ? go<T_Q4_K, 1, DOWN>(a, grid, smem, s) : go<T_Q4_K, 2, DOWN>(a, grid, smem, s);
    case T_Q6_K: return one ? go<T_Q6_K, 1, DOWN>(a, grid, smem, s) : go<T_Q6_K, 2, DOWN>(a, grid, smem, s);
    case T_Q8_0: return one ? go<T_Q8_0, 1, DOWN>(a, grid, smem, s) : go<T_Q8_0, 2, DOWN>(a, grid, smem, s);
    case T_Q5_0: return one ? go<T_Q5_0, 1, DOWN>(a, grid, smem, s) : go<T_Q5_0, 2, DOWN>(a, grid, smem, s);
    case T_Q4_0: return one ? go<T_Q4_0, 1, DOWN>(a, grid, smem, s) : go<T_Q4_0, 2, DOWN>(a, grid, smem, s);
    case T_Q5_K: return one ? go<T_Q5_K, 1, DOWN>(a, grid, smem, s) : go<T_Q5_K, 2, DOWN>(a, grid, smem, s);
    case T_Q2_K: return one ? go<T_Q2_K, 1, DOWN>(a, grid, smem, s) : go<T_Q2_K, 2, DOWN>(a, grid, smem, s);
    case T_Q3_K: return one ? go<T_Q3_K, 1, DOWN>(a, grid, smem, s) : go<T_Q3_K, 2, DOWN>(a, grid, smem, s);
    }
    return cudaErrorInvalidValue;
}

// The two products, each in a file of its own (compiled side by side).
cudaError_t launch_up(int type, Args& a, int sms, cudaStream_t s);
cudaError_t launch_down(int type, Args& a, int sms, cudaStream_t s);

}  // namespace moe
}  // namespace qk
