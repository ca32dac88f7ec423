// qk_moe.cuh -- the products of a mixture-of-experts layer over packed expert
// weights for a few tokens (qk_moe_ffn): g = Wg x and u = Wu x of every (token,
// expert) pair, then y = Wd (SiLU(g) * u).
//
// A decode batch meets few tokens per expert, so the weights of the experts
// met are streamed once, and the work per weight must be small enough for the
// SMs to keep pace.  Pairs are grouped by expert (at most NT, 4 or 8, to a
// group) in every CTA, from the ids alone; a weight is converted once per group
// and multiplied with all its activations (qk_dunits.cuh).
//   * A job is one group, one slice of K (`ku` units of 256) and two tiles of 16
//     rows that share the activations: the gate's and the up's rows (up), or 32
//     rows (down).  Every CTA (one per SM) has a range of jobs, of which its warps
//     take the next one each (fixed turns left the warps of the schedulers with
//     one warp more, and with them the launch, 10 % behind).
//   * A warp streams the packed rows of its jobs into its own two slots of
//     shared memory (cp.async, one step of 256 columns ahead) and waits for
//     nobody else's: with one warp filling stages for eight by bulk copies, the
//     copies (20 to 50 ns each on an SM, whatever their size up to a kilobyte)
//     and the sums of the stage's warps took longer than the products: 61
//     tokens, 8 of 128 experts of 2048 x 768, Q4_K and Q6_K: 374 us a layer,
//     now 169.
//   * Two more warps prepare the activations of the next (group, slice) while
//     the others work on one: x in `up`, SiLU(g) * u in `down` (the first is
//     prepared by all).
//   * Slices of K leave partial sums, added in order by whoever reads them: the
//     preparation of `down`, and a last kernel that also weighs and adds the
//     experts.  The result does not depend on timing.
// What bounds it: 13 tokens, 2 of 8 experts of 4096 x 14336: up 122 us (Q4_K, 529
// MB, 55 % of the DRAM rate), down 135 (Q6_K, 441 MB, 42 %), issue slots half used,
// no pipe above 70 %; with the products left out the layer takes 202 us of its
// 297, with nothing fetched 248, so each side takes the other's place, likely in
// the load-store unit.  One token: some 8 us a product, of which the weights'
// bytes are 2.
#pragma once
#include <algorithm>
#include <cmath>

#include "qk_dunits.cuh"
#include "qk_internal.h"
#include "qk_ptx.cuh"

namespace qk {
namespace moe {

constexpr int kMaxWarps = 14;                         // that multiply (with the two others 16: 128 registers each)
constexpr int kPrepWarps = 2;
constexpr int kMaxThreads = (kMaxWarps + kPrepWarps) * 32;
constexpr int kTileRows = 16;
constexpr int kUnitW = 256;
constexpr uint16_t kNone = 0xffff;

struct Args {
    const float* x;             // up: [n_tok, cols]; down: partial sums of g, then u: [2][slices_in][pairs][cols]
    int slices_in;
    int64_t cols, rows;         // of one expert's matrix
    uint32_t row_bytes;
    const uint8_t *W0, *W1;     // up: gate and up matrices; down: its matrix, twice
    int n_exp, n_tok, k, pairs;
    const int32_t* ids;         // [n_tok, k]
    float* out;                 // up: [2][slices][pairs][rows]; down: [slices][pairs][rows]
    int nxb, nunits;            // of a row: 32-blocks, units
    int ku, slices;             // units of a slice; slices of a row
    int jobs;                   // of a (group, slice)
    int nw;                     // warps that multiply
    int gmax;                   // groups the tables hold
    uint32_t off_pairs, off_gexp, off_gbeg, off_gcnt, off_bar, off_x, off_ring;
    unsigned* status;
    int cap;                    // most pairs of a group (4 or 8)
};

struct Tables {
    uint16_t *pairs, *gexp, *gbeg, *gcnt;   // pairs by expert; expert, first pair and pairs of a group
    int* n;                                 // number of groups
};

// ids (shared, one per pair, kNone = none) -> groups of at most CAP pairs, by
// expert, an expert's pairs in order.  scratch: 3 * n_exp + 1 words, zeroed.  A
// pair's place among its expert's is the number of earlier tokens that chose
// it, from a mask of tokens per expert; given ids may name an expert twice for
// one token: then the pairs are counted one after another.
template <int CAP>
__device__ __forceinline__ void make_groups(const Args& p, const Tables& t, const uint16_t* ids, uint32_t* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, nt = (int)blockDim.x;
    if (p.n_tok == 1) {   // every pair is a group of its own
        if (tid < 32) {
            const bool ok = lane < p.pairs && ids[lane] != kNone;   // at most 16
            const unsigned m = __ballot_sync(0xffffffffu, ok);
            const int at = __popc(m & ((1u << lane) - 1));
            if (ok) {
                t.pairs[at] = (uint16_t)lane;
                t.gexp[at] = ids[lane];
                t.gbeg[at] = (uint16_t)at;
                t.gcnt[at] = 1;
            }
            if (lane == 0) *t.n = __popc(m);
        }
        return;
    }
    uint32_t* mask = scratch;                  // [n_exp][2]: tokens
    uint32_t* offs = scratch + 2 * p.n_exp;    // [n_exp]: first place
    uint32_t* twice = scratch + 3 * p.n_exp;
    for (int i = tid; i < p.pairs; i += nt) {
        const int e = ids[i], tok = i / p.k;
        if (e != kNone && (atomicOr(&mask[2 * e + (tok >> 5)], 1u << (tok & 31)) >> (tok & 31) & 1)) *twice = 1;
    }
    __syncthreads();
    const bool again = *twice != 0;
    if (again) {   // counts in place of masks
        __syncthreads();
        if (tid == 0) {
            for (int e = 0; e < p.n_exp; ++e) mask[2 * e] = mask[2 * e + 1] = 0;
            for (int i = 0; i < p.pairs; ++i)
                if (ids[i] != kNone) ++mask[2 * ids[i]];
        }
        __syncthreads();
    }
    auto count = [&](int e) -> int { return again ? (int)mask[2 * e] : __popc(mask[2 * e]) + __popc(mask[2 * e + 1]); };
    if (tid < 32) {
        // Experts in order, a run of them per lane: running sums of pairs and groups.
        const int per = (p.n_exp + 31) / 32, e0 = lane * per, e1 = min(e0 + per, p.n_exp);
        int np = 0, ng = 0;
        for (int e = e0; e < e1; ++e) {
            np += count(e);
            ng += (count(e) + CAP - 1) / CAP;
        }
        int ip = np, ig = ng;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, ip, o), b = __shfl_up_sync(0xffffffffu, ig, o);
            if (lane >= o) {
                ip += a;
                ig += b;
            }
        }
        if (lane == 31) *t.n = ig;
        ip -= np;
        ig -= ng;
        for (int e = e0; e < e1; ++e) {
            offs[e] = (uint32_t)ip;
            for (int c = count(e); c > 0; c -= CAP) {
                t.gexp[ig] = (uint16_t)e;
                t.gbeg[ig] = (uint16_t)ip;
                t.gcnt[ig] = (uint16_t)min(c, CAP);
                ip += min(c, CAP);
                ++ig;
            }
        }
    }
    __syncthreads();
    if (again) {
        if (tid == 0)
            for (int i = 0; i < p.pairs; ++i)
                if (ids[i] != kNone) t.pairs[offs[ids[i]]++] = (uint16_t)i;
    } else {
        for (int i = tid; i < p.pairs; i += nt) {
            const int e = ids[i], tok = i / p.k;
            if (e == kNone) continue;
            const uint32_t below = (1u << (tok & 31)) - 1;
            const int before = tok < 32 ? __popc(mask[2 * e] & below) : __popc(mask[2 * e]) + __popc(mask[2 * e + 1] & below);
            t.pairs[offs[e] + before] = (uint16_t)i;
        }
    }
}

// Packed rows of a unit in shared memory: 16-byte chunks of a row from the
// boundary at or before its first byte, rows an odd number of chunks apart
// (conflict-free for eight rows at a time).
template <int T>
struct Slot {
    static constexpr int kUB = dm::DU<T>::UB;
    // rows of the 256-weight types with 16-byte blocks start on boundaries, the others on even addresses (Q2_K: on fours)
    static constexpr int kSkew = T == T_Q4_K || T == T_Q5_K ? 0 : T == T_Q2_K ? 12 : 14;
    static constexpr int kChunks = (kUB + kSkew + 15) / 16;
    static constexpr int kRow = 16 * (kChunks | 1);
    static constexpr int kTile = kTileRows * kRow;
    // of a warp: two steps of two tiles, and the scales of a step's
    static constexpr int kWarp = 4 * kTile + (dm::DU<T>::kSc ? 2 * 4 * dm::kScalePitch * 16 : 0);
};

__device__ __forceinline__ void cp_async16_stream(uint32_t dst, const void* src, uint64_t policy, bool on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.u32 q, %3, 0;\n\t"
        "@q cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n\t}" ::"r"(dst),
        "l"(src), "l"(policy), "r"((uint32_t)on)
        : "memory");
}

// A lane's chunks of a tile: numbers lane, lane + 32, .. of its 16 * kChunks,
// row by row (neighbouring lanes read neighbouring chunks); the offsets of
// their rows are kept.
template <int T>
struct Chunks {
    static constexpr int kN = (kTileRows * Slot<T>::kChunks + 31) / 32;
    uint32_t row[kN];   // row * row_bytes
    __device__ __forceinline__ void set(uint32_t rb, int lane) {
#pragma unroll
        for (int i = 0; i < kN; ++i) row[i] = (uint32_t)((lane + 32 * i) / Slot<T>::kChunks) * rb;
    }
    // 16 rows of one unit to dst: `src` is the first byte of row 0's part, `bytes` what each row has of the unit.
    __device__ __forceinline__ void fetch(const uint8_t* src, int bytes, uint32_t dst, int lane, uint64_t pol) const {
        using S = Slot<T>;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int at = lane + 32 * i, r = at / S::kChunks, c16 = 16 * (at - r * S::kChunks);
            const bool in = (kTileRows * S::kChunks) % 32 == 0 || i + 1 < kN || at < kTileRows * S::kChunks;
            const uint8_t* p = src + row[i];
            if (S::kSkew == 0) {
                cp_async16_stream(dst + r * S::kRow + c16, p + c16, pol, in);
            } else {
                const uint32_t skew = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
                cp_async16_stream(dst + r * S::kRow + c16, p - skew + c16, pol, in && c16 < (int)skew + bytes);
            }
        }
    }
};

template <int T, int NT, bool DOWN>
__global__ void __launch_bounds__(kMaxThreads, 1) moe_kernel(const Args p) {
    using U = dm::DU<T>;
    using S = Slot<T>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + p.off_bar);   // [2]: activations prepared
    uint64_t* xfree = xfull + 2;                                       // [2]: no longer used
    volatile int* abort = reinterpret_cast<volatile int*>(xfree + 2);
    Tables tb;
    tb.pairs = reinterpret_cast<uint16_t*>(smem + p.off_pairs);
    tb.gexp = reinterpret_cast<uint16_t*>(smem + p.off_gexp);
    tb.gbeg = reinterpret_cast<uint16_t*>(smem + p.off_gbeg);
    tb.gcnt = reinterpret_cast<uint16_t*>(smem + p.off_gcnt);
    tb.n = const_cast<int*>(reinterpret_cast<volatile int*>(xfree + 2)) + 1;
    int* taken = tb.n + 1;   // jobs that have been handed out
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rb = p.row_bytes;
    // Prepared activations, two sets: B fragments, then block sums.
    const uint32_t x_bytes = (uint32_t)p.ku * NT * dm::kXRow, x_set = x_bytes + (uint32_t)p.ku * 8 * NT * 16;
    uint8_t* xbuf = smem + p.off_x;

    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&xfull[b], kPrepWarps);
            mbar_init(&xfree[b], p.nw);
        }
        *abort = 0;
        *taken = p.nw;
        fence_barrier_init();
    }
    if (DOWN) pdl_launch_dependents();
    {
        uint16_t* ids = reinterpret_cast<uint16_t*>(smem + p.off_ring);   // before the first fetch
        uint32_t* scratch = reinterpret_cast<uint32_t*>(smem + p.off_ring + 2 * ((p.pairs + 7) & ~7));
        if (p.n_tok > 1)
            for (int i = threadIdx.x; i <= 3 * p.n_exp; i += blockDim.x) scratch[i] = 0;
        // `down` is let go by `up` only when that one has seen the kernel before it to its end, so the ids stand for
        // both: `down` makes its groups and asks for its first weights while the last CTAs of `up` still work.
        if (!DOWN) {
            pdl_wait_prior();
            pdl_launch_dependents();
        }
        for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) {
            const int e = __ldcg(p.ids + i);
            ids[i] = e >= 0 && e < p.n_exp ? (uint16_t)e : kNone;
        }
        __syncthreads();
        make_groups<NT>(p, tb, ids, scratch);
        __syncthreads();
    }
    // My jobs: index ((group * slices + slice) * jobs + job), below 2^30.
    const uint32_t total = (uint32_t)*tb.n * p.slices * p.jobs;
    const int each = (int)(total / gridDim.x), more = (int)(total % gridDim.x), bx = (int)blockIdx.x;
    const int j0 = bx * each + min(bx, more), j1 = j0 + each + (bx < more ? 1 : 0);
    if (j0 >= j1) {
        if (DOWN) pdl_wait_prior();   // no grid ends before the one that it follows
        return;
    }
    const int e0 = j0 / p.jobs, e1 = (j1 - 1) / p.jobs;   // my (group, slice)s

    // The activations of (group, slice) e into its set: every step-th (unit, pair) from `first` on, two at a time.
    auto prepare = [&](int e, int first, int step) {
        const int set = (e - e0) & 1, g = e / p.slices, u0 = (e - g * p.slices) * p.ku, nu = min(p.ku, p.nunits - u0);
        const int n = tb.gcnt[g], beg = tb.gbeg[g];
        uint8_t* xb = xbuf + set * x_set;
        float4* xm = reinterpret_cast<float4*>(xb + x_bytes);
#pragma unroll 1
        for (int i0 = first; i0 < nu * n; i0 += 2 * step) {
            float4 a[2], b[2];
            int at[2], un[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int i = min(i0 + m * step, nu * n - 1);
                un[m] = i / n;
                at[m] = i - un[m] * n;
                const int pair = tb.pairs[beg + at[m]], u = u0 + un[m];
                a[m] = b[m] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (8 * u + (lane >> 2) < p.nxb) {
                    const float4* src = reinterpret_cast<const float4*>(
                        p.x + (int64_t)(DOWN ? pair : pair / p.k) * p.cols + (int64_t)u * kUnitW + 8 * lane);
                    if constexpr (!DOWN) {
                        a[m] = __ldcg(src);
                        b[m] = __ldcg(src + 1);
                    } else {
                        const int64_t slice = (int64_t)p.pairs * p.cols / 4, up = slice * p.slices_in;
                        float4 c = a[m], d = a[m];
                        auto add = [](float4& v, float4 w) { v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w; };
#pragma unroll 4
                        for (int k = 0; k < p.slices_in; ++k) {
                            add(a[m], __ldcg(src + k * slice));
                            add(b[m], __ldcg(src + k * slice + 1));
                            add(c, __ldcg(src + up + k * slice));
                            add(d, __ldcg(src + up + k * slice + 1));
                        }
                        auto h = [](float g, float u) { return g / (1.0f + expf(-g)) * u; };   // SiLU(g) u
                        a[m] = make_float4(h(a[m].x, c.x), h(a[m].y, c.y), h(a[m].z, c.z), h(a[m].w, c.w));
                        b[m] = make_float4(h(b[m].x, d.x), h(b[m].y, d.y), h(b[m].z, d.z), h(b[m].w, d.w));
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
                if (i0 + m * step < nu * n)
                    dm::put_x<NT, U::kW4, U::kG16 && (U::kMin || U::kOff != 0), U::kOff>(a[m], b[m], xb + un[m] * (NT * dm::kXRow), xm + un[m] * 8 * NT, at[m], lane);
        }
    };

    // ---------------- multiplies ----------------
    const int g8 = lane >> 2, t = lane & 3;
    const uint64_t pol = policy_evict_first();
    uint8_t* slots = smem + p.off_ring + warp * S::kWarp;
    const uint32_t slots_u32 = smem_u32(slots);
    Chunks<T> chunks;
    chunks.set(rb, lane);
    // A step: one unit of a job.
    struct Step {
        int job, u, end;      // job, unit, and the end of the slice
        int64_t off0, off1;   // byte offsets of the tiles' first rows
    };
    auto enter = [&](Step& s) {   // the first unit of job s.job
        const int e = s.job / p.jobs, j = s.job - e * p.jobs, g = e / p.slices;
        s.u = (e - g * p.slices) * p.ku;
        s.end = min(s.u + p.ku, p.nunits);
        const int64_t row = (int64_t)tb.gexp[g] * p.rows + (int64_t)j * (DOWN ? 2 * kTileRows : kTileRows);
        s.off0 = row * rb;
        s.off1 = DOWN ? s.off0 + (int64_t)kTileRows * rb : s.off0;
    };
    auto fetch = [&](const Step& s, int slot) {
        if (s.job < j1) {
            const int at = s.u * S::kUB;
            const int bytes = min(S::kUB, (int)rb - at);
            chunks.fetch(p.W0 + s.off0 + at, bytes, slots_u32 + slot * (2 * S::kTile), lane, pol);
            chunks.fetch(p.W1 + s.off1 + at, bytes, slots_u32 + slot * (2 * S::kTile) + S::kTile, lane, pol);
        }
        cp_async_commit();
    };
    auto advance = [&](Step& s) {
        if (++s.u < s.end) return;
        int n = 0;
        if (lane == 0) n = atomicAdd(taken, 1);
        s.job = j0 + __shfl_sync(0xffffffffu, n, 0);
        if (s.job < j1) enter(s);
    };
    Step cur, ahead;
    cur.job = warp < p.nw ? j0 + warp : j1;
    if (cur.job < j1) enter(cur);
    ahead = cur;
    fetch(ahead, 0);
    // All warps prepare the first set, then two of them the others while the rest multiplies.  (A set's barriers count
    // its uses: set 0 is full at first without one.)
    if (DOWN) pdl_wait_prior();   // the sums of `up`
    prepare(e0, warp, p.nw + kPrepWarps);
    __syncthreads();
    if (warp >= p.nw) {
        for (int e = e0 + 1; e <= e1; ++e) {
            const int set = (e - e0) & 1, turn = (e - e0) >> 1;
            if (turn > 0 && !mbar_wait_abortable(&xfree[set], (uint32_t)(turn - 1) & 1u, p.status, abort)) return;
            prepare(e, warp - p.nw, kPrepWarps);
            __syncwarp();
            if (lane == 0) mbar_arrive(&xfull[set]);
        }
        return;
    }
    int slot = 0, e = e0 - 1;   // e: the activations in use
    bool dead = false;
    // Leaves the activations up to those before `to` (in their order: a set is free when every warp has left it).
    auto leave = [&](int to) {
        for (; e < to && !dead; ++e) {
            if (e >= e0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&xfree[(e - e0) & 1]);
            }
            const int next = e + 1 - e0, fill = (next >> 1) - (next & 1 ? 0 : 1);   // the set's fill that a barrier counts
            if (e + 1 <= e1 && next > 0 && !mbar_wait_abortable(&xfull[next & 1], (uint32_t)fill & 1u, p.status, abort)) dead = true;
        }
    };
    while (cur.job < j1 && !dead) {
        const int me = cur.job / p.jobs, j = cur.job - me * p.jobs, g = me / p.slices, u0 = cur.u;
        float2 ya[NT / 4] = {}, yb[NT / 4] = {};
        leave(me);
        if (dead) break;
        const uint8_t* xb = xbuf + ((me - e0) & 1) * x_set;
        const float4* xm = reinterpret_cast<const float4*>(xb + x_bytes);
        for (int u = u0; u < cur.end; ++u) {
            if (ahead.job < j1) advance(ahead);
            fetch(ahead, slot ^ 1);
            cp_async_wait<1>();
            __syncwarp();   // every lane's chunks of this step have arrived
            const uint8_t* q = slots + slot * (2 * S::kTile) + g8 * S::kRow;
            const uint32_t at = (uint32_t)u * S::kUB, o0 = (uint32_t)cur.off0 + at, o1 = (uint32_t)cur.off1 + at;
            const uint8_t* a0 = q + ((o0 + g8 * rb) & 15u);
            const uint8_t* a1 = q + 8 * S::kRow + ((o0 + (g8 + 8) * rb) & 15u);
            const uint8_t* b0 = q + S::kTile + ((o1 + g8 * rb) & 15u);
            const uint8_t* b1 = q + S::kTile + 8 * S::kRow + ((o1 + (g8 + 8) * rb) & 15u);
            dm::run_unit<T, NT>(a0, a1, b0, b1, xb + (u - u0) * (NT * dm::kXRow), xm + (u - u0) * 8 * NT,
                                reinterpret_cast<float4*>(slots + 4 * S::kTile), lane, min(8, p.nxb - 8 * u), ya, yb);
            __syncwarp();   // every lane is done with the slot
            slot ^= 1;
        }
        // The job's sums of the group's pairs.
        const int n = tb.gcnt[g], beg = tb.gbeg[g], sl = me - g * p.slices;
        const int64_t stack = (int64_t)p.slices * p.pairs * p.rows;
#pragma unroll
        for (int k = 0; k < NT / 4; ++k) {
            const int i = NT == 4 ? t : 2 * t + k;
            if (i < n) {
                float* o = p.out + ((int64_t)sl * p.pairs + tb.pairs[beg + i]) * p.rows + (int64_t)j * (DOWN ? 2 * kTileRows : kTileRows) + g8;
                o[0] = ya[k].x;
                o[8] = ya[k].y;
                float* o2 = DOWN ? o + kTileRows : o + stack;
                o2[0] = yb[k].x;
                o2[8] = yb[k].y;
            }
        }
        cur = ahead;
    }
    if (!dead) leave(e1);
    cp_async_wait<0>();
}

// ------------------------------------------------------------------- host --
constexpr int64_t kSmemMax = 227 * 1024;

// Shared memory handed out piece by piece.
struct Take {
    int64_t at = 0;
    uint32_t operator()(int64_t bytes) {
        const int64_t o = at;
        at = (at + bytes + 15) & ~(int64_t)15;
        return (uint32_t)o;
    }
};

// Groups that n tokens make of n_exp experts if each chooses k of them at
// random, at most cap pairs to a group.
inline double groups_of(int n, int k, int n_exp, int cap) {
    const double p = (double)k / n_exp;
    if (p >= 1.0) return (double)n_exp * ((n + cap - 1) / cap);
    double sum = 0.0, c = std::pow(1.0 - p, n);   // probability of exactly i tokens
    for (int i = 0; i <= n; ++i) {
        sum += c * ((i + cap - 1) / cap);
        c *= (double)(n - i) / (i + 1) * p / (1.0 - p);
    }
    return n_exp * sum;
}

// The geometry of one product: the size of groups (cap: 4 or 8; 0 where nothing fits) and the
// slices of K that are expected to take the least time, in units' times: a job
// costs its units (1.25 each with groups of eight, for their second B loads and
// MMAs) and 0.7 for its sums and their way out.  warp_bytes of shared memory for
// two steps of a warp.
// The four numbers in it are fitted to times; both sides of each choice, with one
// product's geometry forced (the layer, us; narrow: 8 of 128 experts of 2048 x 768,
// wide: 2 of 8 of 4096 x 14336, Q4_K and Q6_K):
//   groups of 4 / 8: 13 tokens narrow 94 / 101 (up), 94 / 102 (down), wide 289 / 299
//     (up), 289 / 289 (down); 61 narrow 169 / 170, 168 / 171; 64 wide 852 / 738, 858 / 737;
//   units of a slice of up, 1 / 2 / 4 / 8: 61 narrow 187 / 171 / 169 / 170, 13 wide
//     346 / 312 / 291 / 289, 64 wide 876 / 780 / 737 / 852 (fours again);
//   of down, 1 / 2 / 3 / 4 / 6: 13 wide 311 / 290 / 285 / 289 / 300, 64 wide 801 / 738 /
//     729 / 727 / 879.  (The planned 2 there makes 28 slices, whose partial sums,
//     59 MB, are not counted: 1.5 %.)
// One token: 28 and 69, the best of all 28 and 68.
inline void plan(Args& a, int type_block_bytes, int type_block_elems, int warp_bytes, bool down, int sms, uint32_t* smem) {
    a.row_bytes = (uint32_t)(a.cols / type_block_elems * type_block_bytes);
    a.nxb = (int)(a.cols / 32);
    a.nunits = (int)((a.cols + kUnitW - 1) / kUnitW);
    a.jobs = (int)(a.rows / (down ? 2 * kTileRows : kTileRows));
    double best = 1e300;
    Args chosen = a;
    chosen.cap = 0;
    for (const int cap : {4, 8}) {
        if (cap == 8 && a.n_tok <= 4) continue;
        const double groups = groups_of(a.n_tok, a.k, a.n_exp, cap);
        for (const int most : {8, 7, 6, 5, 4, 3, 2, 1}) {
            Args b = a;
            b.slices = (a.nunits + most - 1) / most;
            b.ku = (a.nunits + b.slices - 1) / b.slices;
            b.slices = (a.nunits + b.ku - 1) / b.ku;
            b.gmax = std::min(a.pairs, a.n_exp + a.pairs / cap);
            Take take;
            b.off_pairs = take(2 * a.pairs);
            b.off_gexp = take(2 * b.gmax);
            b.off_gbeg = take(2 * b.gmax);
            b.off_gcnt = take(2 * b.gmax);
            b.off_bar = take(4 * 8 + 16);
            b.off_x = take(2 * (int64_t)b.ku * cap * (dm::kXRow + 8 * 16));
            b.off_ring = (uint32_t)((take.at + 127) & ~(int64_t)127);
            // the last words of a row's reads may lie behind it
            b.nw = (int)std::min<int64_t>((kSmemMax - b.off_ring - 16) / warp_bytes, kMaxWarps);
            if (b.nw < 4) continue;
            // jobs of a warp, and half a job that the last ones to finish take longer
            const double jobs = groups * b.slices * b.jobs / sms / b.nw, turns = jobs > 1.0 ? jobs + 0.5 : 1.0;
            // the SM's issue slots are shared by its warps; a dozen of them use what there is
            const double time = turns * std::max(b.nw, 12) * (b.ku * (cap == 4 ? 1.0 : 1.25) + 0.7);
            if (time < best) {
                best = time;
                const int64_t ring = std::max<int64_t>((int64_t)b.nw * warp_bytes, 2 * ((a.pairs + 7) & ~7) + 12 * a.n_exp + 16);
                *smem = (uint32_t)(b.off_ring + ring + 16);
                chosen = b;
                chosen.cap = cap;
            }
        }
    }
    a = chosen;
}

template <class K>
cudaError_t launch_kernel(K kern, const Args& a, int grid, uint32_t smem, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)(a.nw + kPrepWarps) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int T, int BB, int BE, bool DOWN>
cudaError_t go(Args& a, int sms, cudaStream_t s, bool launch) {
    uint32_t smem = 0;
    plan(a, BB, BE, Slot<T>::kWarp, DOWN, sms, &smem);
    if (a.cap == 0) return cudaErrorInvalidValue;
    if (!launch) return cudaSuccess;
    return a.cap == 4 ? launch_kernel(moe_kernel<T, 4, DOWN>, a, sms, smem, s) : launch_kernel(moe_kernel<T, 8, DOWN>, a, sms, smem, s);
}

template <bool DOWN>
cudaError_t launch_product(int type, Args& a, int sms, cudaStream_t s, bool launch) {
    switch (type) {
    case T_Q4_K: return go<T_Q4_K, 144, 256, DOWN>(a, sms, s, launch);
    case T_Q6_K: return go<T_Q6_K, 210, 256, DOWN>(a, sms, s, launch);
    case T_Q8_0: return go<T_Q8_0, 34, 32, DOWN>(a, sms, s, launch);
    case T_Q5_0: return go<T_Q5_0, 22, 32, DOWN>(a, sms, s, launch);
    case T_Q4_0: return go<T_Q4_0, 18, 32, DOWN>(a, sms, s, launch);
    case T_Q5_K: return go<T_Q5_K, 176, 256, DOWN>(a, sms, s, launch);
    case T_Q2_K: return go<T_Q2_K, 84, 256, DOWN>(a, sms, s, launch);
    case T_Q3_K: return go<T_Q3_K, 110, 256, DOWN>(a, sms, s, launch);
    }
    return cudaErrorInvalidValue;
}

// The two products, in files of their own (compiled side by side).  launch
// false: only the geometry (slices).
cudaError_t launch_up(int type, Args& a, int sms, cudaStream_t s, bool launch);
cudaError_t launch_down(int type, Args& a, int sms, cudaStream_t s, bool launch);

}  // namespace moe
}  // namespace qk
