// qk_tree.cu -- attention of drafted-token trees over the paged, block-
// quantized KV cache, on the tcgen05 tensor cores.
//
// For token i of request r, query head h and its kv head g:
//   s_t = scale q_h . K[t, g] over the visible t,  out = sum softmax(s)_t V[t, g].
//
// All tokens and heads that share a kv head read the same cache rows, so a
// unit of work is (request, kv head, up to 64 rows), a row being a (token,
// head of the group).  A unit's positions are walked in tiles of BN (128; 64
// for d = 256); the tiles of all units form one list, cut into equal runs, one
// per CTA (persistent, one CTA per SM), so ragged lengths balance and one long
// request fills the GPU.  A unit cut between CTAs leaves partial sums that
// join_kernel combines (log-sum-exp, in order): deterministic.
//
// Both products have the positions (or d) as their 128-row side and the rows
// as N, which costs what the rows need (N = 16 .. 64) instead of 128:
//   S^T [positions x rows] = K [positions x d] Q^T     A = K, B = Q, K-major
//   O^T [d x rows]        += V^T [d x positions] P     A = V, B = P, MN-major
// K and V tiles are decoded once per unit to fp16 (code * d, one rounding) and
// serve both as they lie, [position][d] in 128-byte swizzled rows; no
// transposition anywhere.  A softmax thread owns one position and all rows of
// a tile.  Row maxima are needed only as a reference: a tile keeps the
// present reference unless some score exceeds it by 2^8 (one vote), and only
// then the new maxima are found and O and the sums are rescaled, so the
// ordinary tile has no reduction across threads; the rows' sums of
// probabilities stay per thread until the unit's end.
//
// Warps: 0 copies (cp.async.bulk of the pages' contiguous head slabs into a
// ring), 1 issues the MMAs, 2-3 load the unit's queries, 4-7 softmax and
// epilogue (TMEM lanes), 8-15 decode.  Every hand-over is an mbarrier with a
// bounded wait; after a wait has run out (status word) the copies and MMAs
// stop, the other roles run through without waiting, and the CTA leaves in
// order.
//
// What is not visible never reaches a result: a masked score is replaced, not
// added to; rows past the end are decoded as zeros; a V block whose scale is
// not finite is decoded as zero and recorded, and the epilogue sets NaN for the
// rows that do see it.  A V tile with values past fp16's range (scales up to
// 65504 times a code of 128 are legal) is decoded times 2^-7 and summed apart
// (O^T's second set of columns), which the epilogue adds times 2^7.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "qk_formats.cuh"
#include "qk_hunits.cuh"
#include "qk_internal.h"
#include "qk_paged.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace tree {

constexpr int kRows = 64;        // rows of a unit, at most (N of the MMAs)
constexpr int kDq = 8;           // decoding warps
constexpr int kThreads = (8 + kDq) * 32;
constexpr int kH = 3;            // fp16 tile buffers (K and V tiles alternate)
constexpr int kTmem = 512;       // columns: S^T twice 64, O^T 128 (two halves of d = 256), the same for large V tiles
constexpr int kTmemO = 128, kTmemBig = 256;
constexpr float kBig = 128.0f;   // scale of the large V tiles
constexpr float kLift = 7.0f;    // probabilities are held times 2^7 (fp16 keeps 2^-21 of the maximum at full precision)
constexpr float kOver = 15.0f;   // and stay below 2^15

struct Args {
    const __nv_bfloat16* q;
    int64_t n_tok, q_stride;
    const uint8_t *K, *V;
    Pool pool;
    const int32_t* table;
    int64_t table_stride;
    const int32_t *ctx, *cu;
    const uint64_t* mask;
    int n_req, max_q, G, n_heads;
    float scale;
    __nv_bfloat16* out;
    int64_t out_stride;
    uint8_t* ws;
    int ctas;
    unsigned* status;
};

struct Req {
    int64_t tok0;
    int64_t ctx;
    int n;
};
__device__ __forceinline__ Req req_of(const Args& a, int r) {
    Req q;
    q.tok0 = min(max((int64_t)a.cu[r], (int64_t)0), a.n_tok);
    q.n = (int)min(max(min((int64_t)a.cu[r + 1], a.n_tok) - q.tok0, (int64_t)0), (int64_t)a.max_q);
    q.ctx = max(a.ctx[r], 0);
    return q;
}
// The drafted tokens that token i of the request sees.
__device__ __forceinline__ uint64_t seen_of(const Args& a, const Req& q, int i) {
    const uint64_t in = q.n >= 64 ? ~uint64_t(0) : (uint64_t(1) << q.n) - 1;
    return (a.mask ? a.mask[q.tok0 + i] : (i >= 63 ? ~uint64_t(0) : (uint64_t(2) << i) - 1)) & in;
}

// Geometry of one instantiation.
template <int T, int D> struct Geo {
    static constexpr int BN = D == 256 ? 64 : 128;         // positions per tile
    static constexpr int NB = D / 32;                      // blocks per row
    static constexpr int RB = NB * Fmt<T>::BB;             // bytes per row
    static constexpr int CH = D <= 64 ? 1 : D / 64;        // 64-element chunks of a row
    static constexpr int CHB = BN * 128;                   // bytes of a chunk: BN rows of 128
    static constexpr int HB = CH * CHB;                    // an fp16 tile
    static constexpr int QB = CH * kRows * 128;            // the unit's queries
    static constexpr int PB = BN * 128;                    // one P tile
    static constexpr int RAW = BN * RB + 16;               // a packed tile
    static constexpr int SEGS = BN * D / 64;               // 64-element segments of a tile
    static constexpr int SPW = D <= 64 ? 32 : 2048 / D;    // segments across, per decoding warp
    static constexpr int PPS = D == 32 ? 2 : 1;            // positions per segment
    static constexpr int FIXED = kH * HB + QB + 2 * PB;
    static constexpr int MISC = 8192;
    static constexpr int NS0 = (227 * 1024 - 1024 - MISC - FIXED) / RAW;
    static constexpr int NS = NS0 > 8 ? 8 : NS0;           // ring stages
    static constexpr int SMEM = 1024 + FIXED + NS * RAW + MISC;
    static_assert(NS >= 2 && RAW % 16 == 0, "tree attention's ring");
    // A partial result: O [rows][D], reference and sum per row.
    static constexpr int64_t PART = (int64_t)kRows * (D + 2) * 4;
};

struct __align__(16) Misc {
    float cmul[kRows];           // scale * log2 e * 2^e of the row's query
    float cref[kRows];           // kLift less the row's reference
    uint64_t seen[4][kRows];     // by unit mod 4
    float colc[4][kRows];
    uint4 valid[16];             // by tile mod 16: bit per position that exists
    float ref[kRows], factor[kRows];
    float wsum[4][kRows];
    int wmax[4][kRows];
    unsigned long long bad_draft[4][8];   // by unit mod 4, 32-block: drafted V rows that are not finite
    unsigned bad_ctx[4][8];
    unsigned big_tile[16];       // by tile mod 16: the V tile is decoded times 2^-7
    unsigned used[4];            // by unit mod 4: bit 0 the plain sums, bit 1 the large tiles' sums hold something
    uint64_t raw_full[8], raw_empty[8], h_full[kH], h_empty[kH], s_full[2], s_empty[2], p_full[2], pv_done[2];
    uint64_t q_full, q_empty, o_empty, drain;
    long long scan[16];
    long long start_base;
    int start_r, abort;
    uint32_t tmem;
};
static_assert(sizeof(Misc) <= 8192, "Misc");

// ------------------------------------------------------- the work list ----

__device__ __forceinline__ int tiles_of(const Req& q, int bn) { return (int)((q.ctx + q.n + bn - 1) / bn); }
__device__ __forceinline__ int groups_of(const Req& q, int G) { return (q.n * G + kRows - 1) / kRows; }
__device__ __forceinline__ int64_t work_of(const Args& a, const Req& q, int bn) {
    return q.n ? (int64_t)a.pool.n_kv * groups_of(q, a.G) * tiles_of(q, bn) : 0;
}
// Columns (N of the MMAs) a unit of that many rows takes.
__device__ __forceinline__ int cols_of(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

struct Piece {
    Req q;
    int r, g, row0, rows;    // the unit: request, kv head, its rows
    int t0, t1, nt;          // tiles [t0, t1) of its nt
    int64_t u0;              // place of its tile 0 in the work list
};
// The pieces of the run [x, end) of the list, from request r whose tiles
// start at base.
struct Walk {
    int64_t x, end, base;
    int r;
    __device__ __forceinline__ bool next(const Args& a, int bn, Piece& p) {
        if (x >= end) return false;
        Req q = req_of(a, r);
        int64_t w = work_of(a, q, bn);
        while (x >= base + w) {
            base += w;
            q = req_of(a, ++r);
            w = work_of(a, q, bn);
        }
        const int nt = tiles_of(q, bn), gr = groups_of(q, a.G);
        const int64_t rel = x - base;
        const int unit = (int)(rel / nt);
        p.q = q;
        p.r = r;
        p.g = unit / gr;
        p.row0 = (unit - p.g * gr) * kRows;
        p.rows = min(kRows, q.n * a.G - p.row0);
        p.nt = nt;
        p.t0 = (int)(rel - (int64_t)unit * nt);
        p.t1 = (int)min((int64_t)nt, p.t0 + (end - x));
        p.u0 = x - p.t0;
        x += p.t1 - p.t0;
        return true;
    }
};

// What a cut unit leaves for join_kernel, per CTA boundary: the unit that
// starts in the previous CTA and reaches into this one (rows == 0: none).
struct __align__(16) Cut {
    int rows, first, last;   // rows; CTAs of its first and last piece
    int first_slot;          // 2 c + (0: the piece starts at the CTA's run, 1: later)
    long long tok0;
    int row0, g;
};

// ------------------------------------------------------------- PTX bits ----

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Packed fp32 pairs (each half rounded as by itself).
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 unpair(uint64_t v) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Barrier of the four softmax warps; true where any of their threads asks.
__device__ __forceinline__ bool vote_softmax(bool any) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)any)
        : "memory");
    return r != 0;
}
// The same of the eight decoding warps.
__device__ __forceinline__ bool vote_decode(bool any) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 2, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)any)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_softmax() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor: fp16 A and B (format 0), fp32 D, M = 128; bits 15
// and 16 mark A and B as MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool mn) {
    return (1u << 4) | (mn ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
// MN-major operand in 128-byte swizzled rows (a row: 64 elements of the MN
// side at one k): stride byte offset 1024 from 8 k to the next 8, leading
// byte offset from 64 MN elements to the next 64.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t smem_addr, uint32_t mn_stride) {
    return (tc::sdesc_k128(smem_addr) & ~(uint64_t(0x3FFF) << 16)) | ((uint64_t)((mn_stride >> 4) & 0x3FFFu) << 16);
}

// bulk_g2s without a cache hint, for bytes that other units read again.
__device__ __forceinline__ void bulk_g2s_keep(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// A wait of the roles that run on after a failure: no waiting once *abort is set.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, unsigned* status, volatile int* abort) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1; i < kWaitSpins; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if ((i & 63u) == 0 && globaltimer_ns() - t0 > kWaitNs) break;
    }
    *abort = 1;
    atomicOr(status, STATUS_TIMEOUT);
    return false;
}
// The same for a whole warp: one lane polls, the others wait for it.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Args& a, volatile int* abort) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0 && !mbar_try_wait(bar, parity)) ok = wait_long(bar, parity, a.status, abort);
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// --------------------------------------------------------------- decode ----
// fp16 code * d (one rounding), in 16-byte chunks of eight.  The codes are
// taken two at a time out of each word by a mask, which puts a 32-block's
// elements in the order
//   Q8_0:        chunk k = 8 k + {0, 2, 1, 3, 4, 6, 5, 7},
//   Q4_0, Q5_0:  chunk k = 4 k + {0, 2, 1, 3}, 16 + 4 k + {0, 2, 1, 3};
// the queries are laid out in the same order and the epilogue undoes it.
template <int T>
__device__ __forceinline__ int element_of(int slot) {
    const int k = slot >> 3, j = slot & 7, p = (j & 4) | ((j & 1) << 1) | ((j >> 1) & 1);
    return T == T_Q8_0 ? 8 * k + p : 4 * k + (p & 3) + ((p & 4) << 2);
}

// Largest code magnitude.
template <int T> __host__ __device__ constexpr float code_max() { return T == T_Q8_0 ? 128.0f : (T == T_Q5_0 ? 16.0f : 8.0f); }

// A segment is 64 elements, two blocks: 17, 9 or 11 words from a 4-byte
// aligned shared address (rows are whole segments, except that at d = 32 a
// segment is two rows).
template <int T> struct Seg {
    static constexpr int BYTES = 2 * Fmt<T>::BB, W = BYTES / 4;
    uint32_t w[W];
    __device__ __forceinline__ explicit Seg(const uint8_t* p) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = hm::lds32(p + 4 * i);
    }
    // Scale bits of block b (0, 1); word i past block b's scale.
    __device__ __forceinline__ uint32_t scale(int b) const { return b ? w[Fmt<T>::BB / 4] >> 16 : w[0] & 0xffffu; }
    __device__ __forceinline__ uint32_t word(int b, int i) const {
        return b ? w[(Fmt<T>::BB + 2) / 4 + i] : __funnelshift_r(w[i], w[i + 1], 16);
    }
    // Chunk k (0..3) of block b: code (exact) * d; a large tile takes the
    // code times 2^-7, still exact.
    template <bool BIG>
    __device__ __forceinline__ uint4 chunk(int b, int k, uint32_t d2) const {
        using hm::and_or;
        using hm::and_xor;
        using hm::hadd2;
        const auto value = [d2](uint32_t code) { return hmul2(BIG ? hmul2(code, 0x20002000u) : code, d2); };
        if constexpr (T == T_Q8_0) {   // 0x6480 ^ byte = 1152 + (signed byte)
            const uint32_t x = word(b, 2 * k), y = word(b, 2 * k + 1);
            return make_uint4(value(hadd2(and_xor(x, 0x00FF00FFu, 0x64806480u), 0xE480E480u)),
                              value(hadd2(and_xor(x >> 8, 0x00FF00FFu, 0x64806480u), 0xE480E480u)),
                              value(hadd2(and_xor(y, 0x00FF00FFu, 0x64806480u), 0xE480E480u)),
                              value(hadd2(and_xor(y >> 8, 0x00FF00FFu, 0x64806480u), 0xE480E480u)));
        } else if constexpr (T == T_Q4_0) {   // low nibbles 1024 + q - 1032, high ones 64 + q - 72
            const uint32_t x = word(b, k), y = x >> 8;
            return make_uint4(value(hadd2(and_or(x, 0x000F000Fu, 0x64006400u), 0xE408E408u)),
                              value(hadd2(and_or(y, 0x000F000Fu, 0x64006400u), 0xE408E408u)),
                              value(hadd2(and_or(x, 0x00F000F0u, 0x54005400u), 0xD480D480u)),
                              value(hadd2(and_or(y, 0x00F000F0u, 0x54005400u), 0xD480D480u)));
        } else {   // the fifth bits of 4 elements spread to bit 4 of their bytes; 1024 + q - 1040
            const uint32_t qh = word(b, 0), x = word(b, 1 + k);
            const uint32_t lo = (x & 0x0F0F0F0Fu) | ((((qh >> (4 * k)) & 15u) * 0x02040810u) & 0x10101010u);
            const uint32_t hi = ((x >> 4) & 0x0F0F0F0Fu) | ((((qh >> (16 + 4 * k)) & 15u) * 0x02040810u) & 0x10101010u);
            return make_uint4(value(hadd2(and_or(lo, 0x00FF00FFu, 0x64006400u), 0xE410E410u)),
                              value(hadd2(and_or(lo >> 8, 0x00FF00FFu, 0x64006400u), 0xE410E410u)),
                              value(hadd2(and_or(hi, 0x00FF00FFu, 0x64006400u), 0xE410E410u)),
                              value(hadd2(and_or(hi >> 8, 0x00FF00FFu, 0x64006400u), 0xE410E410u)));
        }
    }
};

// -------------------------------------------------------------- softmax ----

// Sums over the warp of v[0 .. 16 NC): lane l gets the sums of columns l (and
// l + 32) in v[0] (and v[1]), by exchanging halves.
template <int NC>
__device__ __forceinline__ void warp_sums(float (&v)[16 * NC], int lane) {
    constexpr int C = 16 * NC;
    if constexpr (C == 16) {   // a 32-wide exchange starts with the two halves adding up
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const bool up = lane & o;
                const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
    } else {
#pragma unroll
        for (int h = 0; h < C; h += 32)
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const bool up = lane & o;
                    const float give = up ? v[h + i] : v[h + i + o], keep = up ? v[h + i + o] : v[h + i];
                    v[h + i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        if constexpr (C == 64) v[1] = v[32];
    }
}

// One piece of a unit by the softmax warps, with 16 NC columns (rows) live.
// tile: running count of the CTA's tiles; unit: of its pieces.
template <int T, int D, int NC>
__device__ __forceinline__ void softmax_piece(const Args& a, Misc& m, uint8_t* sp, uint32_t tmem, const Piece& p, uint32_t& tile,
                                              uint32_t unit, uint8_t* part) {
    using G = Geo<T, D>;
    constexpr int C = 16 * NC;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, tid = 32 * wq + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16);
    const uint64_t* seen = m.seen[unit & 3];
    volatile int* abort = &m.abort;
    uint64_t l2[C / 2];   // this thread's sums of probabilities, columns in pairs
#pragma unroll
    for (int c = 0; c < C / 2; ++c) l2[c] = 0;
#pragma unroll 1
    for (int t = p.t0; t < p.t1; ++t, ++tile) {
        const uint32_t b = tile & 1, ph = (tile >> 1) & 1;
        wait_warp(&m.s_full[b], ph, a, abort);
        tc::fence_after_sync();
        uint32_t s[C];
#pragma unroll
        for (int h = 0; h < C; h += 16) tc::tmem_ld16(lanes + 64 * b + h, *reinterpret_cast<uint32_t(*)[16]>(&s[h]));
        const int64_t pos0 = (int64_t)t * G::BN, pos = pos0 + tid;
        const uint4 vw = m.valid[tile & 15];
        const uint32_t mine = wq == 0 ? vw.x : wq == 1 ? vw.y : wq == 2 ? vw.z : vw.w;
        const bool here = (mine >> lane) & 1;   // the position exists (false past BN)
        const bool all = pos0 + G::BN <= p.q.ctx && (vw.x & vw.y) == 0xffffffffu &&
                         (G::BN == 64 || (vw.z & vw.w) == 0xffffffffu);
        const int64_t j = pos - p.q.ctx;   // drafted token at this position, if >= 0
        // Visibility of this position to column c.
        auto vis = [&](int c) { return here && (j < 0 || ((seen[c] >> (j & 63)) & 1)); };
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.s_empty[b]);   // S^T has been read
        const bool first = t == p.t0;
        // log2 of the lifted probabilities of columns c .. c + 3
        auto logs = [&](int c, float (&x)[4]) {
            const float4 k = *reinterpret_cast<const float4*>(&m.cmul[c]), r = *reinterpret_cast<const float4*>(&m.cref[c]);
            const float2 u = unpair(fma2(pair(s[c], s[c + 1]), pair(k.x, k.y), pair(r.x, r.y)));
            const float2 v = unpair(fma2(pair(s[c + 2], s[c + 3]), pair(k.z, k.w), pair(r.z, r.w)));
            x[0] = u.x, x[1] = u.y, x[2] = v.x, x[3] = v.y;
        };
        bool over = first;
        if (!first) {
            float mx = -INFINITY;
            if (all) {
#pragma unroll
                for (int c = 0; c < C; c += 4) {
                    float x[4];
                    logs(c, x);
                    mx = fmaxf(fmaxf(mx, fmaxf(x[0], x[1])), fmaxf(x[2], x[3]));
                }
            } else {
#pragma unroll
                for (int c = 0; c < C; c += 4) {
                    float x[4];
                    logs(c, x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, vis(c + i) ? x[i] : -INFINITY);
                }
            }
            over = mx > kOver && (G::BN == 128 || tid < G::BN);
        }
        if (vote_softmax(over)) {
            // New references: the rows' maxima over the tile, as ordered integers.
            const float* mul = m.colc[unit & 3];
#pragma unroll
            for (int h = 0; h < C; h += 16) {
                int keep = 0;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    float y = __uint_as_float(s[h + c]) * mul[h + c];
                    if (!(vis(h + c) && y == y)) y = -INFINITY;
                    int k = __float_as_int(y);
                    k ^= (k >> 31) & 0x7fffffff;
                    k = __reduce_max_sync(0xffffffffu, k);
                    if (lane == c) keep = k;
                }
                if (lane < 16) m.wmax[wq][h + lane] = keep;
            }
            sync_softmax();
            if (tid < C) {
                int k = max(max(m.wmax[0][tid], m.wmax[1][tid]), max(m.wmax[2][tid], m.wmax[3][tid]));
                k ^= (k >> 31) & 0x7fffffff;
                const float old = first ? -INFINITY : m.ref[tid], now = fmaxf(old, __int_as_float(k));
                m.factor[tid] = old == -INFINITY ? 0.0f : ex2(old - now);
                m.ref[tid] = now;
                m.cmul[tid] = mul[tid];
                m.cref[tid] = kLift - now;
            }
            sync_softmax();
            if (!first) {
#pragma unroll
                for (int c = 0; c < C; c += 2) l2[c / 2] = mul2(l2[c / 2], *reinterpret_cast<const uint64_t*>(&m.factor[c]));
                wait_warp(&m.pv_done[b ^ 1], ((tile - 1) >> 1) & 1, a, abort);   // O^T is at rest
                tc::fence_after_sync();
                const bool big = *(volatile unsigned*)&m.used[unit & 3] & 2;
#pragma unroll 1
                for (int h = 0; h < (big ? 2 : 1) * (D == 256 ? 2 : 1) * C; h += 16) {
                    const int set = h / C, c0 = h - set * C;   // D = 256: halves, then the large tiles' halves
                    const uint32_t at = lanes + (D == 256 ? kTmemO + 64 * set : set ? kTmemBig : kTmemO) + c0;
                    uint32_t v[16];
                    tc::tmem_ld16(at, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * m.factor[c0 + c]);
                    tmem_st16(at, v);
                }
                tmem_wait_st();
            }
        }
        if (tile >= 2) wait_warp(&m.pv_done[b], ((tile >> 1) - 1) & 1, a, abort);   // the P buffer is free
        uint8_t* row = sp + b * G::PB + tid * 128;
        // Probabilities of columns c .. c + 7 into the position's row.
        auto eight = [&](int c, auto masked) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                float x[4];
                logs(c + i, x);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = ex2(x[k]);
                    if constexpr (decltype(masked)::value) x[k] = vis(c + i + k) ? x[k] : 0.0f;
                }
                l2[(c + i) / 2] = add2(l2[(c + i) / 2], pair(x[0], x[1]));
                l2[(c + i) / 2 + 1] = add2(l2[(c + i) / 2 + 1], pair(x[2], x[3]));
                o[i / 2] = pack_f16(x[0], x[1]);
                o[i / 2 + 1] = pack_f16(x[2], x[3]);
            }
            if (G::BN == 128 || tid < G::BN)
                *reinterpret_cast<uint4*>(row + (((c / 8) ^ (tid & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        };
        if (all) {
#pragma unroll
            for (int c = 0; c < C; c += 8) eight(c, std::false_type{});
        } else {
#pragma unroll
            for (int c = 0; c < C; c += 8) eight(c, std::true_type{});
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_full[b]);
    }
    float l[C];
#pragma unroll
    for (int c = 0; c < C; c += 2) {
        const float2 u = unpair(l2[c / 2]);
        l[c] = u.x;
        l[c + 1] = u.y;
    }
    // Epilogue: the rows' sums over the threads, then O^T.
    if (G::BN == 64 && tid >= 64)
#pragma unroll
        for (int c = 0; c < C; ++c) l[c] = 0.0f;   // threads past BN held no position
    warp_sums<NC>(l, lane);
    if (lane < C) m.wsum[wq][lane] = l[0];
    if constexpr (C == 64) m.wsum[wq][32 + lane] = l[1];
    const uint32_t last = tile - 1;
    wait_warp(&m.pv_done[last & 1], (last >> 1) & 1, a, abort);
    tc::fence_after_sync();
    sync_softmax();
    const bool whole = p.t0 == 0 && p.t1 == p.nt;
    const unsigned used = *(volatile unsigned*)&m.used[unit & 3];
    float* po = reinterpret_cast<float*>(part);
    float* pm = po + kRows * D;
    if (!whole && tid < p.rows) {
        pm[2 * tid] = -m.cref[tid];
        pm[2 * tid + 1] = m.wsum[0][tid] + m.wsum[1][tid] + m.wsum[2][tid] + m.wsum[3][tid];
    }
#pragma unroll 1
    for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
        const int blk = 4 * half + wq;
        if (blk >= G::NB) break;   // lanes past d (warp-uniform)
        const int e = 32 * blk + element_of<T>(lane);
        const uint64_t bad = m.bad_draft[unit & 3][blk];
        const bool badc = m.bad_ctx[unit & 3][blk] != 0;
#pragma unroll 1
        for (int h = 0; h < C; h += 16) {
            uint32_t v[16];
            tc::tmem_ld16(lanes + kTmemO + 64 * half + h, v);
            tc::tmem_wait_ld();
            if (used != 1) {
                uint32_t u[16];
                tc::tmem_ld16(lanes + kTmemBig + 64 * half + h, u);
                tc::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    v[c] = __float_as_uint((used & 1 ? __uint_as_float(v[c]) : 0.0f) + (used & 2 ? kBig * __uint_as_float(u[c]) : 0.0f));
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const int col = h + c;
                if (col >= p.rows) continue;
                float o = __uint_as_float(v[c]);
                if (badc || (bad & seen[col])) o = __int_as_float(0x7fffffff);
                if (whole) {
                    const float sum = m.wsum[0][col] + m.wsum[1][col] + m.wsum[2][col] + m.wsum[3][col];
                    const int row = p.row0 + col, tok = row / a.G;
                    a.out[(p.q.tok0 + tok) * a.out_stride + (p.g * a.G + row - tok * a.G) * D + e] =
                        __float2bfloat16_rn(sum == 0.0f ? 0.0f : __fdividef(o, sum));
                } else {
                    po[col * D + e] = o;
                }
            }
        }
        __syncwarp();
        if (lane == 0) {
            m.bad_draft[unit & 3][blk] = 0;
            m.bad_ctx[unit & 3][blk] = 0;
        }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&m.o_empty);
}

// --------------------------------------------------------------- kernel ----

template <int T, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const Args a) {
    using G = Geo<T, D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sh = smem;                 // fp16 tiles
    uint8_t* sq = sh + kH * G::HB;      // queries
    uint8_t* sp = sq + G::QB;           // P
    uint8_t* raw = sp + 2 * G::PB;      // packed tiles
    Misc& m = *reinterpret_cast<Misc*>(raw + G::NS * G::RAW);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Cut* cuts = reinterpret_cast<Cut*>(a.ws);
    uint8_t* parts = a.ws + (int64_t)a.ctas * sizeof(Cut);

    pdl_launch_dependents();
    if (warp == 1) {
        tc::tmem_alloc(&m.tmem, kTmem);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < G::NS; ++i) {
            mbar_init(&m.raw_full[i], 1);
            mbar_init(&m.raw_empty[i], kDq);
        }
        for (int i = 0; i < kH; ++i) {
            mbar_init(&m.h_full[i], kDq);
            mbar_init(&m.h_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.s_full[i], 1);
            mbar_init(&m.s_empty[i], 4);
            mbar_init(&m.p_full[i], 4);
            mbar_init(&m.pv_done[i], 1);
        }
        mbar_init(&m.q_full, 2);
        mbar_init(&m.q_empty, 1);
        mbar_init(&m.o_empty, 4);
        mbar_init(&m.drain, 1);
        m.abort = 0;
        m.start_r = -1;
        fence_barrier_init();
    }
    if (tid < 32) {
        m.bad_draft[tid >> 3][tid & 7] = 0;
        m.bad_ctx[tid >> 3][tid & 7] = 0;
    }
    // The list's length, then the request that holds this CTA's first tile.
    int64_t total = 0, per = 0, x0 = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        int64_t carry = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < a.n_req; r0 += kThreads) {
            const int r = r0 + tid;
            const int64_t w = r < a.n_req ? work_of(a, req_of(a, r), G::BN) : 0;
            int64_t v = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            __syncthreads();
            if (lane == 31) m.scan[warp] = v;
            __syncthreads();
            int64_t before = carry, sum = carry;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) {
                if (i < warp) before += m.scan[i];
                sum += m.scan[i];
            }
            if (pass == 1 && before + v - w <= x0 && x0 < before + v) {
                m.start_r = r;
                m.start_base = before + v - w;
            }
            carry = sum;
        }
        total = carry;
        per = (total + a.ctas - 1) / a.ctas;
        x0 = (int64_t)blockIdx.x * per;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = m.tmem;
    const int64_t x1 = min(x0 + per, total);
    const bool works = x0 < x1;
    const Walk begin{x0, works ? x1 : x0, works ? m.start_base : 0, works ? m.start_r : 0};
    volatile int* abort = &m.abort;

    if (tid == 0) {   // the cut at this CTA's start
        Cut c{};
        Walk w = begin;
        Piece p;
        if (w.next(a, G::BN, p) && p.t0 > 0) {
            const int first = (int)(p.u0 / per);
            if (first == (int)blockIdx.x - 1) {
                c.rows = p.rows;
                c.first = first;
                c.last = (int)((p.u0 + p.nt - 1) / per);
                c.first_slot = 2 * first + (p.u0 % per != 0);
                c.tok0 = p.q.tok0;
                c.row0 = p.row0;
                c.g = p.g;
            }
        }
        cuts[blockIdx.x] = c;
    }
    __syncwarp();

    // Registers: 80 + 176 + 2 x 128 per thread of the four warpgroups, the launch's 4 x 128.
    if (warp >= 4 && warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        Walk w = begin;
        Piece p;
        uint32_t tile = 0, unit = 0;
#pragma unroll 1
        for (; w.next(a, G::BN, p); ++unit) {
            uint8_t* part = parts + (2 * (int64_t)blockIdx.x + (p.t0 == 0 && p.u0 != x0)) * G::PART;
            if (p.rows <= 16) softmax_piece<T, D, 1>(a, m, sp, tmem, p, tile, unit, part);
            else if (p.rows <= 32) softmax_piece<T, D, 2>(a, m, sp, tmem, p, tile, unit, part);
            else softmax_piece<T, D, 4>(a, m, sp, tmem, p, tile, unit, part);
        }
    } else if (warp >= 8) {
        // Decode: a thread takes one segment.  A warp's lanes are SPW
        // positions by 32 / SPW segments of the row, so that its word loads
        // fall into 32 different banks (a row's segments are 17, 9 or 11 words
        // apart, odd; positions 1, 2 or 4 times that) and eight neighbouring
        // lanes' 16-byte stores into the eight bank groups of swizzled rows.
        Walk w = begin;
        Piece p;
        uint32_t n = 0, tile = 0, unit = 0;
        const int dt = tid - 256;
        static_assert(G::SEGS <= kDq * 32, "a segment per decoding thread");
        const bool mine = dt < G::SEGS;
        const int pos0 = mine ? ((dt / 32) * G::SPW + lane % G::SPW) * G::PPS : 0, seg0 = mine ? lane / G::SPW : 0;
#pragma unroll 1
        for (; w.next(a, G::BN, p); ++unit) {
#pragma unroll 1
            for (int t = p.t0; t < p.t1; ++t, ++tile) {
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int st = n % G::NS, hs = n % kH;
                    wait_warp(&m.raw_full[st], (n / G::NS) & 1, a, abort);
                    if (n >= kH) wait_warp(&m.h_empty[hs], (n / kH - 1) & 1, a, abort);
                    const uint32_t* valid = reinterpret_cast<const uint32_t*>(&m.valid[tile & 15]);
                    const Seg<T> seg(raw + st * G::RAW + pos0 * G::RB + seg0 * Seg<T>::BYTES);
                    uint32_t db[2];
                    bool good[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int pos = pos0 + (D == 32 ? i : 0);
                        db[i] = seg.scale(i);
                        good[i] = mine && ((valid[pos >> 5] >> (pos & 31)) & 1);
                    }
                    bool big = false;
                    if (kv) {   // V: scales that are not finite, or too large for fp16 times a code
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float d = fabsf(h2f(db[i]));
                            if (good[i] && !(d * code_max<T>() <= 65504.0f)) {
                                big = big || d <= 65504.0f;
                                if (!(d <= 65504.0f)) {
                                    const int64_t j = (int64_t)t * G::BN + pos0 + (D == 32 ? i : 0) - p.q.ctx;
                                    const int blk = D == 32 ? 0 : 2 * seg0 + i;
                                    if (j < 0) atomicOr(&m.bad_ctx[unit & 3][blk], 1u);
                                    else atomicOr(&m.bad_draft[unit & 3][blk], 1ull << (j & 63));
                                    good[i] = false;
                                }
                            }
                        }
                        big = vote_decode(big);
                        if (dt == 0) m.big_tile[tile & 15] = big;
                    }
                    if (mine) {
                        auto blocks = [&](auto is_big) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int pos = pos0 + (D == 32 ? i : 0);
                                uint8_t* line = sh + hs * G::HB + seg0 * G::CHB + pos * 128;
                                const uint32_t d2 = hm::dup16(db[i]);
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    uint4 o = seg.template chunk<decltype(is_big)::value>(i, k, d2);
                                    if (!good[i]) o = make_uint4(0, 0, 0, 0);
                                    *reinterpret_cast<uint4*>(line + ((((D == 32 ? 0 : 4 * i) + k) ^ (pos & 7)) << 4)) = o;
                                }
                            }
                        };
                        if (big) blocks(std::true_type{});
                        else blocks(std::false_type{});
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&m.raw_empty[st]);
                        mbar_arrive(&m.h_full[hs]);
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 0) {
            // Copies: the tile's rows of every page it touches, K then V.
            Walk w = begin;
            Piece p;
            uint32_t n = 0, tile = 0;   // stages requested, tiles
            const uint64_t pol = policy_evict_first();
            bool ok = true;
            const int page = 1 << a.pool.page_log2, span = min(page, G::BN), slabs = G::BN / span;
            while (ok && w.next(a, G::BN, p)) {
                const int64_t len = p.q.ctx + p.q.n;
                const bool shared = groups_of(p.q, a.G) > 1;   // other row groups read these bytes too
                const int32_t* tab = a.table + (int64_t)p.r * a.table_stride;
#pragma unroll 1
                for (int t = p.t0; ok && t < p.t1; ++t, ++tile) {
                    const int64_t pos0 = (int64_t)t * G::BN, pos = pos0 + (int64_t)lane * span;
                    const bool live = lane < slabs && pos < len;
                    int id = -1;
                    if (live) id = page_of(a.pool, tab, a.table_stride, pos, a.status);
                    const unsigned have = __ballot_sync(0xffffffffu, id >= 0);
                    const int rows = live && id >= 0 ? (int)min((int64_t)span, len - pos) : 0;
                    const uint32_t bytes = (uint32_t)(rows * G::RB + 15) & ~15u;   // whole slabs are multiples of 16
                    const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes);
                    // Lane L reports positions 4 L .. 4 L + 3, which lie in one page.
                    uint32_t bits = 0;
                    if (4 * lane < G::BN && ((have >> (4 * lane / span)) & 1)) {
                        const int64_t left = len - (pos0 + 4 * lane);
                        bits = left >= 4 ? 15u : left > 0 ? (1u << left) - 1 : 0u;
                    }
                    bits <<= 4 * (lane & 7);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
                    if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(&m.valid[tile & 15])[lane >> 3] = bits;
                    __syncwarp();   // the valid words, before the arrival that publishes them
                    const int64_t off = id >= 0 ? pool_row(a.pool, id, p.g, (int)(pos & (page - 1))) : 0;
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++n) {
                        const int st = n % G::NS;
                        if (n >= G::NS && !wait_warp(&m.raw_empty[st], (n / G::NS - 1) & 1, a, abort)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&m.raw_full[st], sum);
                        __syncwarp();
                        uint8_t* dst = raw + st * G::RAW + lane * span * G::RB;
                        const uint8_t* src = (kv ? a.V : a.K) + off;
                        if (bytes) {
                            if (shared) bulk_g2s_keep(dst, src, bytes, &m.raw_full[st]);
                            else bulk_g2s(dst, src, bytes, &m.raw_full[st], pol);
                        }
                    }
                }
            }
            // Copies in flight land before the CTA may leave.
            if (!ok)
                for (uint32_t i = n > G::NS ? n - G::NS : 0; i < n; ++i)
                    mbar_wait_bounded(&m.raw_full[i % G::NS], (i / G::NS) & 1, a.status);
        } else if (warp == 1) {
            // MMAs: the warp walks together, one lane issues.
            Walk w = begin;
            Piece p;
            uint32_t tile = 0, unit = 0;
            bool ok = true;
            const bool leader = tc::elect_one();
            int n_prev = 0;          // N of the pending P V product; 0: none
            bool first_prev = false; // it is its unit's first
            uint32_t unit_prev = 0;
            unsigned used = 0;       // Misc::used of the pending product's unit
            const uint64_t dk = tc::sdesc_k128(smem_u32(sh)), dq = tc::sdesc_k128(smem_u32(sq));
            // d <= 64: one chunk only, read twice (rows 64 .. 127 of O^T are not used)
            const uint64_t dv = sdesc_mn128(smem_u32(sh), D <= 64 ? 0 : G::CHB), dp = sdesc_mn128(smem_u32(sp), 0);
            uint32_t hs = 0, hph = 0;    // buffer and phase of the next K or V tile
            auto next_h = [&] {
                if (++hs == kH) hs = 0, hph ^= 1;
            };
            uint32_t vs = 0, vph = 0;    // of the pending product's V tile
            auto pv = [&](uint32_t i) {
                const uint32_t b = i & 1;
                ok = ok && wait_warp(&m.h_full[vs], vph, a, abort) && wait_warp(&m.p_full[b], (i >> 1) & 1, a, abort);
                if (first_prev && unit_prev > 0) ok = ok && wait_warp(&m.o_empty, (unit_prev - 1) & 1, a, abort);
                if (!ok) return;
                tc::fence_after_sync();
                const bool big = *(volatile unsigned*)&m.big_tile[i & 15] != 0;
                const unsigned bit = big ? 2u : 1u;
                if (first_prev) used = 0;
                const bool fresh = !(used & bit);
                used |= bit;
                const uint32_t o = big ? kTmemBig : kTmemO, id = idesc_f16(n_prev, true);
                const uint64_t da = dv + (uint64_t)(vs * (G::HB >> 4)), db = dp + (uint64_t)(b * (G::PB >> 4));
                if (leader) {
                    *(volatile unsigned*)&m.used[unit_prev & 3] = used;
#pragma unroll
                    for (int half = 0; half < (D == 256 ? 2 : 1); ++half)
#pragma unroll
                        for (int k = 0; k < G::BN / 16; ++k)
                            tc::mma_bf16(tmem + o + 64 * half, da + (half * (G::CHB >> 3) + 128 * k), db + 128 * k, id,
                                         !fresh || k > 0);
                    tc::commit(&m.h_empty[vs]);
                    tc::commit(&m.pv_done[b]);
                }
                __syncwarp();
            };
            while (ok && w.next(a, G::BN, p)) {
                const int N = cols_of(p.rows);
                const uint32_t id = idesc_f16(N, false);
#pragma unroll 1
                for (int t = p.t0; ok && t < p.t1; ++t, ++tile) {
                    const uint32_t b = tile & 1;
                    ok = ok && wait_warp(&m.h_full[hs], hph, a, abort);
                    if (t == p.t0) ok = ok && wait_warp(&m.q_full, unit & 1, a, abort);
                    if (tile >= 2) ok = ok && wait_warp(&m.s_empty[b], ((tile >> 1) - 1) & 1, a, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint64_t da = dk + (uint64_t)(hs * (G::HB >> 4));
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc::mma_bf16(tmem + 64 * b, da + ((k >> 2) * (G::CHB >> 4) + 2 * (k & 3)),
                                         dq + ((k >> 2) * (kRows * 8) + 2 * (k & 3)), id, k > 0);
                        tc::commit(&m.h_empty[hs]);
                        tc::commit(&m.s_full[b]);
                        if (t == p.t1 - 1) tc::commit(&m.q_empty);
                    }
                    __syncwarp();
                    next_h();
                    if (n_prev) pv(tile - 1);
                    vs = hs;
                    vph = hph;
                    next_h();
                    n_prev = N;
                    first_prev = t == p.t0;
                    unit_prev = unit;
                }
                ++unit;
            }
            if (ok && n_prev) pv(tile - 1);
            if (!ok) {   // let the products in flight end
                if (leader) tc::commit(&m.drain);
                __syncwarp();
                if (lane == 0) mbar_wait_bounded(&m.drain, 0, a.status);
                __syncwarp();
            }
        } else {
            // Queries: row by row to fp16 times a power of two that brings the
            // row's largest magnitude to 2^14 .. 2^15 (bf16's 8 bits are exact).
            Walk w = begin;
            Piece p;
            uint32_t unit = 0;
            constexpr int LPR = D / 8, RPW = 32 / LPR;   // lanes per row, rows per pass
            const int sub = lane % LPR;
#pragma unroll 1
            for (; w.next(a, G::BN, p); ++unit) {
                if (unit > 0) wait_warp(&m.q_empty, (unit - 1) & 1, a, abort);
                const int N = cols_of(p.rows);
#pragma unroll 4
                for (int i = (warp - 2) * RPW + lane / LPR; i < N; i += 2 * RPW) {   // N and the stride are multiples of RPW
                    const bool live = i < p.rows;
                    const int row = p.row0 + i, tok = live ? row / a.G : 0, h = live ? row - tok * a.G : 0;
                    const __nv_bfloat16* q = a.q + (p.q.tok0 + tok) * a.q_stride + (int64_t)(p.g * a.G + h) * D;
                    uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);   // four bf16 each
                    const int b = sub >> 2, k = sub & 3;                  // 32-block, chunk
                    if (live) {
                        if constexpr (T == T_Q8_0) {
                            const uint4 u = *reinterpret_cast<const uint4*>(q + 32 * b + 8 * k);
                            lo = make_uint2(u.x, u.y);
                            hi = make_uint2(u.z, u.w);
                        } else {
                            lo = *reinterpret_cast<const uint2*>(q + 32 * b + 4 * k);
                            hi = *reinterpret_cast<const uint2*>(q + 32 * b + 16 + 4 * k);
                        }
                    }
                    const uint32_t u[4] = {lo.x, lo.y, hi.x, hi.y};
                    float f[8], mx = 0.0f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        f[2 * c] = __uint_as_float(u[c] << 16);
                        f[2 * c + 1] = __uint_as_float(u[c] & 0xffff0000u);
                        mx = fmaxf(mx, fmaxf(fabsf(f[2 * c]), fabsf(f[2 * c + 1])));
                    }
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    int ex = (int)(__float_as_uint(mx) >> 23) - 127 - 14;   // mx < 2^(ex + 15)
                    if (mx == 0.0f || ex > 113) ex = 0;                       // nothing, or not finite
                    ex = max(ex, -126);                                       // the factors stay normal
                    const float down = __uint_as_float((uint32_t)(127 - ex) << 23), up = __uint_as_float((uint32_t)(127 + ex) << 23);
                    uint4 o;   // slots 0, 2, 1, 3, ... of the loaded order
                    o.x = pack_f16(f[0] * down, f[2] * down);
                    o.y = pack_f16(f[1] * down, f[3] * down);
                    o.z = pack_f16(f[4] * down, f[6] * down);
                    o.w = pack_f16(f[5] * down, f[7] * down);
                    *reinterpret_cast<uint4*>(sq + (sub >> 3) * (kRows * 128) + i * 128 + (((sub & 7) ^ (i & 7)) << 4)) = o;
                    if (sub == 0) {
                        m.colc[unit & 3][i] = live ? a.scale * 1.44269504088896341f * up : 0.0f;
                        m.seen[unit & 3][i] = live ? seen_of(a, p.q, tok) : 0;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.q_full);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmem);
    }
}

// Joins the pieces of the units that were cut: block (c, y) takes rows y, y +
// gridDim.y, ... (one per warp) of the unit cut at CTA c's start.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Args a) {
    constexpr int E = D / 32;
    pdl_wait_prior();
    const Cut c = reinterpret_cast<const Cut*>(a.ws)[blockIdx.x];
    const uint8_t* parts = a.ws + (int64_t)a.ctas * sizeof(Cut);
    constexpr int64_t PART = (int64_t)kRows * (D + 2) * 4;
    const int lane = threadIdx.x & 31;
    for (int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); row < c.rows; row += gridDim.y * kJoinWarps) {
        auto part = [&](int i) {   // piece i, 0 .. last - first
            return reinterpret_cast<const float*>(parts + (i == 0 ? c.first_slot : 2 * (int64_t)(c.first + i)) * PART);
        };
        const int n = c.last - c.first + 1;
        float top = -INFINITY;
        for (int i = lane; i < n; i += 32) top = fmaxf(top, part(i)[kRows * D + 2 * row]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.0f, acc[E] = {};
        for (int i0 = 0; i0 < n; i0 += 32) {
            float f = 0.0f, lf = 0.0f;   // this lane's piece: its factor, its share of the sum
            if (i0 + lane < n) {
                const float* pm = part(i0 + lane) + kRows * D + 2 * row;
                // a piece that saw nothing has sum 0 (and no reference)
                f = pm[1] == 0.0f ? 0.0f : ex2(pm[0] - top);
                lf = pm[1] == 0.0f ? 0.0f : f * pm[1];
            }
#pragma unroll 4
            for (int i = 0; i < 32 && i0 + i < n; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                sum += __shfl_sync(0xffffffffu, lf, i);
                const float* po = part(i0 + i) + row * D + lane;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += fi * po[32 * e];
            }
        }
        const int rr = c.row0 + row, tok = rr / a.G;
        __nv_bfloat16* o = a.out + (c.tok0 + tok) * a.out_stride + (int64_t)(c.g * a.G + rr - tok * a.G) * D + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) o[32 * e] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc[e] / sum);
    }
}

template <int T, int D>
static cudaError_t launch_t(const Args& a, cudaStream_t s) {
    using G = Geo<T, D>;
    cudaError_t e = cudaFuncSetAttribute(tree_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e != cudaSuccess) return e;
    tree_kernel<T, D><<<a.ctas, kThreads, G::SMEM, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas, kRows / kJoinWarps);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, a);
}
template <int T>
static cudaError_t launch_d(const Args& a, int d, cudaStream_t s) {
    switch (d) {
    case 32: return launch_t<T, 32>(a, s);
    case 64: return launch_t<T, 64>(a, s);
    case 128: return launch_t<T, 128>(a, s);
    case 256: return launch_t<T, 256>(a, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tree

// The grid: one CTA per SM, fewer when the call cannot have that many tiles.
static int tree_ctas(int64_t n_req, int max_q, int64_t max_pos, int n_heads, int n_kv, int d, int sms) {
    const int bn = d == 256 ? 64 : 128;
    const double tiles = (double)n_req * n_kv * (((int64_t)max_q * (n_heads / n_kv) + tree::kRows - 1) / tree::kRows) *
                         ((max_pos + bn - 1) / bn);
    return tiles < sms ? std::max(1, (int)tiles) : sms;
}

int64_t attn_tree_ws_bytes(int64_t n_req, int max_q, int64_t max_pos, int n_heads, int n_kv, int d, int sms) {
    const int ctas = tree_ctas(n_req, max_q, max_pos, n_heads, n_kv, d, sms);
    return ctas * ((int64_t)sizeof(tree::Cut) + 2 * (int64_t)tree::kRows * (d + 2) * 4);
}

cudaError_t launch_attn_tree(int type, const void* q, int64_t n_tok, int64_t q_stride, const uint8_t* K, const uint8_t* V,
                             int64_t n_pages, int page_log2, int row_bytes, const int32_t* table, int64_t table_stride,
                             const int32_t* ctx, const int32_t* cu, const uint64_t* mask, int64_t n_req, int max_q,
                             int n_heads, int n_kv, int d, float scale, void* out, int64_t out_stride, void* ws,
                             unsigned* status, int sms, cudaStream_t s) {
    const tree::Args a{static_cast<const __nv_bfloat16*>(q), n_tok, q_stride, K, V, Pool{n_pages, page_log2, n_kv, row_bytes},
                       table, table_stride, ctx, cu, mask, (int)n_req, max_q, n_heads / n_kv, n_heads, scale,
                       static_cast<__nv_bfloat16*>(out), out_stride, static_cast<uint8_t*>(ws),
                       tree_ctas(n_req, max_q, table_stride << page_log2, n_heads, n_kv, d, sms), status};
    switch (type) {
    case T_Q8_0: return tree::launch_d<T_Q8_0>(a, d, s);
    case T_Q5_0: return tree::launch_d<T_Q5_0>(a, d, s);
    case T_Q4_0: return tree::launch_d<T_Q4_0>(a, d, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace qk
