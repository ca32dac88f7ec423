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
//   S^T [positions x rows] = K [positions x d] Q^T     A = K from tensor memory, B = Q
//   O^T [d x rows]        += V^T [d x positions] P     A = V, B = P, MN-major in shared memory
// K and V tiles are decoded once per unit to fp16 (code * d, one rounding): K
// straight into tensor memory, a lane per position; V as it lies, [position]
// [d] in 128-byte swizzled rows.  No transposition anywhere.  A softmax thread
// owns one position and half of the rows of a tile.  Row maxima are needed
// only as a reference: a tile keeps the present reference unless some score
// exceeds it by 2^8 (one vote), and only then the new maxima are found and O
// and the sums are rescaled, so the ordinary tile has no reduction across
// threads; the rows' sums of probabilities are one more product, with ones in
// V's place, which leaves them in every lane.
//
// Warps: 0 and 3 copy K and V (cp.async.bulk of the pages' contiguous head
// slabs into a ring), 1 issues Q K, 2 issues P V; 4-11 softmax and epilogue
// (two warpgroups, half of the rows each); 12-19 decode K; 20-27 decode V and
// load the unit's queries.  A tile is a chain of short steps, so it is the
// number of warps on it that sets the rate: with one warpgroup each for
// softmax and (K and V) decoding a tile took 5,000 clocks.  Every hand-over
// is an mbarrier with a bounded wait (2 s); after a wait has run out (status
// word) the copies and MMAs stop, the other roles run through without waiting
// and without storing results, what is in flight ends, and the CTA leaves in
// order.
//
// What is not visible never reaches a result: a masked score is replaced, not
// added to; rows past the end are decoded as zeros; a V block whose scale is
// not finite is decoded as zero and recorded, and the epilogue sets NaN for the
// rows that do see it.  V blocks with values past fp16's range (scales up to
// 65504 times a code of 128 are legal) are decoded times 2^-7, as a V tile of
// their own with zeros in the other blocks' place, and summed apart (O^T's
// second set of columns), which the epilogue adds times 2^7; the tile of the
// other blocks has zeros in theirs.  So a large block, hidden or not, leaves
// the others' bits alone, and a tile without one costs nothing more.
//
// Roundings to fewer than 32 bits, besides the bf16 output: a cached value
// (code * d has up to 19 bits) and a probability are fp16, 11 bits, because they
// are operands of the tensor cores, whose next wider type has half the rate and
// takes twice the memory (shared memory is full); probabilities are lifted by
// 2^7 so that those down to 2^-21 of the reference keep all 11 bits.
// Scores, references, sums and O are fp32.  Relative to the 64-bit result the
// error is 1.70e-3 to 1.72e-3 over the measured calls; rounding that result
// to bf16 alone gives 1.66e-3 to 1.67e-3.
//
// Bounds and measurements (GB300, GPU time of a call in a replayed graph).  The
// floor is the cache's bytes up to 80 (Q4_0) to 150 (Q8_0) rows a kv head, the
// tensor rate above.  64 requests of 500 to 15,000 positions, Q8_0, 4 to 8
// tokens, 32 / 8 heads of 128 (1.04 GB): 306 us, 3.41 TB/s, 50 % of the measured
// copy rate; one request of 32,765 positions, 16 tokens (71 MB): 45 us, 24 %; 27
// ragged Q4_0 requests in pages of 16 (121 MB): 111 us, 16 %; 64-token trees, 8
// heads to a kv head, Q5_0, d = 64 (12.4 GFLOP): 104 us; one token over 212
// positions: 11.7 us.  A copy of an earlier build (46, 114, 110 and 308 us) without
// decoding, softmax and products, only timed, took 33, 92, 60 and 192 us for the
// four large ones, so copies and hand-overs are more than half of each.  A further
// tile of a long request costs its CTA 1.45 us; in a trace 15,000 clocks passed
// from a unit's last tile to the next unit's first.  Issue slots used while an SM
// was active: 62 % (second case), 74 % (first: 1,935 instructions a scheduler and
// tile, the ALU pipe 52 %), without local spills.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qk_formats.cuh"
#include "qk_hunits.cuh"
#include "qk_internal.h"
#include "qk_paged.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace tree {

constexpr int kThreads = 28 * 32;
constexpr int kSm = 4, kKd = 12, kVd = 20;   // first warps of softmax, K and V decoding
constexpr int kDw = 8;                       // warps of each of these
constexpr int kV = 2;                        // V tile buffers
// Tensor memory: S^T twice 64 columns, O^T 64 (or two halves of 32 at d = 256), the large V blocks' O^T, K twice d / 2.
constexpr int kTmem = 512, kTmemO = 128, kTmemBig = 192, kTmemK = 256;
constexpr float kBig = 128.0f;   // scale of the large V blocks
constexpr float kLift = 7.0f;    // probabilities are held times 2^7 (fp16 keeps 2^-21 of the maximum at full precision)
constexpr float kOver = 15.0f;   // and stay below 2^15
constexpr int kRows = 64;        // most rows of a unit

struct Args {
    const __nv_bfloat16* q;
    int64_t n_tok, q_stride;
    const uint8_t *K, *V;
    Pool pool;
    const int32_t* table;
    int64_t table_stride;
    const int32_t *ctx, *cu;
    const uint64_t* mask;
    int n_req, max_q, G;
    uint32_t g_magic;   // ceil(2^19 / G): row / G = row * g_magic >> 19 for row < 4160, G <= 64
    float scale;
    __nv_bfloat16* out;
    int64_t out_stride;
    uint8_t* ws;
    int ctas;
    unsigned* status;
    uint32_t looks;     // limit of a wait for V's copies, in looks of kTreeLookNs (kTreeLooks but in a test)
    uint32_t hold;      // tile at which a CTA's V copies stop (a test's; ordinarily none)
};

// A request: its first token's row, its tokens, its committed positions and
// the positions walked (those past the table's end, or past QK_TREE_MAX_POS, do not
// exist: they are reported, and not walked).
struct Req {
    int tok0, n, ctx, len;
};
__device__ __forceinline__ Req req_of(const Args& a, int r) {
    Req q;
    const int n_tok = (int)a.n_tok;
    q.tok0 = min(max(a.cu[r], 0), n_tok);
    q.n = min(max(min(a.cu[r + 1], n_tok) - q.tok0, 0), a.max_q);
    const int64_t ctx = max(a.ctx[r], 0), cap = min(a.table_stride << a.pool.page_log2, (int64_t)QK_TREE_MAX_POS);
    q.ctx = (int)min(ctx, cap);
    q.len = (int)min(ctx + q.n, cap);
    if (q.n > 0 && ctx + q.n > cap) atomicOr(a.status, STATUS_BAD_PAGE);
    return q;
}
// The drafted tokens that token i of the request sees.
__device__ __forceinline__ uint64_t seen_of(const Args& a, const Req& q, int i) {
    const uint64_t in = q.n >= 64 ? ~uint64_t(0) : (uint64_t(1) << q.n) - 1;
    return (a.mask ? a.mask[q.tok0 + i] : (i >= 63 ? ~uint64_t(0) : (uint64_t(2) << i) - 1)) & in;
}

// Token of a row: row / G.
__device__ __forceinline__ int token_of(const Args& a, int row) { return (int)((uint32_t)row * a.g_magic >> 19); }

// Geometry of one instantiation.
template <int T, int D> struct Geo {
    static constexpr int BN = D == 256 ? 64 : 128;         // positions per tile
    static constexpr int NR = D == 256 ? 32 : 64;          // rows of a unit, at most
    static constexpr int NB = D / 32;                      // blocks per row
    static constexpr int RB = NB * Fmt<T>::BB;             // bytes per row
    static constexpr int CH = D <= 64 ? 1 : D / 64;        // 64-element chunks of a row
    static constexpr int CHB = BN * 128;                   // bytes of a chunk: BN rows of 128
    static constexpr int VB = CH * CHB;                    // a V tile
    static constexpr int QB = CH * NR * 128;               // the unit's queries
    static constexpr int PB = BN * 128;                    // one P tile
    static constexpr int RAW = BN * RB;                    // a packed tile
    static constexpr int ITEM = D == 32 ? 32 : 64;         // elements a decoding thread takes at once
    static constexpr int ITEMS = BN * D / ITEM;            // of them in a tile
    static constexpr int KC = D / 2;                       // tensor-memory columns of a K tile
    static constexpr int TL = D == 256 ? 32 : 384;         // tensor-memory column of the rows' sums (S^T has 32 columns of 64 at d = 256)
    static constexpr int FIXED = kV * VB + QB + 2 * PB + 1024;   // and the tile of ones
    static constexpr int MISC = 10752;
    static constexpr int NS0 = (227 * 1024 - 1024 - MISC - FIXED) / RAW;
    static constexpr int NS = (NS0 > 8 ? 8 : NS0) & ~1;    // ring stages; even: V tiles always take the odd ones
    static constexpr int SMEM = 1024 + FIXED + NS * RAW + MISC;
    static_assert(NS >= 4 && RAW % 16 == 0, "tree attention's ring");
};
// A partial result: O [rows][D], reference and sum per row.
template <int D> __host__ __device__ constexpr int64_t part_bytes() { return (int64_t)kRows * (D + 2) * 4; }

// A piece of a unit: request, kv head, rows (0: no more pieces), tiles [t0,
// t1) of nt.  One warp walks the list and hands the pieces to the others
// through shared memory, so that their divisions are done once and take no
// registers elsewhere.
struct __align__(16) Piece {
    Req q;
    int r, g, row0, rows, t0, t1, nt, u0;   // u0: place of its tile 0 in the work list
};

struct __align__(16) Misc {
    float cmul[kRows];           // scale * log2 e * 2^e of the row's query
    float cref[kRows];           // kLift less the row's reference
    uint64_t seen[4][kRows];     // by unit mod 4, as the next two
    float colc[4][kRows];
    int64_t rowoff[4][kRows];    // the row's place in out, -1 for columns that are no row
    uint4 valid[2][16];          // K's, V's copier: by tile mod 16, a bit per position that exists
    float ref[kRows], factor[kRows];
    float wmax[4][kRows];
    unsigned long long bad_draft[8][8];   // by unit mod 8, 32-block: drafted V rows that are not finite
    unsigned bad_ctx[8][8];
    unsigned big_tile[16];       // by tile mod 16: the V tile is followed by one of its large blocks
    unsigned used[8];            // by unit mod 8: whether the large blocks' sums hold something
    uint64_t raw_full[8], raw_empty[8], k_full[2], k_empty[2], v_full[kV], v_empty[kV], s_full[2],
        p_full[2], pv_done[2];
    uint64_t q_full, q_empty, o_empty, big_full, big_empty, drain[2], piece_full[8], piece_free[8];
    Piece piece[8];              // by unit mod 8
    int scan[32];
    Req start_q;
    int start_base, start_w, start_r, abort;
    uint32_t tmem;
};
static_assert(sizeof(Misc) <= 10752, "Misc");

// ------------------------------------------------------- the work list ----
// Counts of tiles stay inside 31 bits (the host refuses more).

__device__ __forceinline__ int tiles_of(const Req& q, int bn) { return (q.len + bn - 1) / bn; }
__device__ __forceinline__ int groups_of(const Req& q, int G, int nr) { return (q.n * G + nr - 1) / nr; }
template <int BN, int NR> __device__ __forceinline__ int work_of(const Args& a, const Req& q) {
    return q.n ? a.pool.n_kv * groups_of(q, a.G, NR) * max(tiles_of(q, BN), 1) : 0;
}
// Columns (N of the MMAs) a unit of that many rows takes.
__device__ __forceinline__ int cols_of(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// The pieces of the run [x, end) of the list; the present request r's tiles
// start at base.
template <int BN, int NR> struct Walk {
    int x, end, base, w, r;   // w: the present request's tiles
    Req q;
    __device__ __forceinline__ bool next(const Args& a, Piece& p) {
        if (x >= end) return false;
        while (x >= base + w) {
            base += w;
            q = req_of(a, ++r);
            w = work_of<BN, NR>(a, q);
        }
        const int nt = max(tiles_of(q, BN), 1), gr = groups_of(q, a.G, NR);
        const int rel = x - base, unit = rel / nt;
        p.r = r;
        p.g = unit / gr;
        p.row0 = (unit - p.g * gr) * NR;
        p.rows = min(NR, q.n * a.G - p.row0);
        p.nt = nt;
        p.t0 = rel - unit * nt;
        p.t1 = min(nt, p.t0 + (end - x));
        p.u0 = x - p.t0;
        p.q = q;
        x += p.t1 - p.t0;
        return true;
    }
};

// What a cut unit leaves for join_kernel, per CTA boundary: the unit that
// starts in the previous CTA and reaches into this one (rows == 0: none).
struct __align__(16) Cut {
    int rows, first, last;   // rows; CTAs of its first and last piece
    int first_slot;          // 2 c + (0: the piece starts at the CTA's run, 1: later)
    int tok0, row0, g, pad;
};

// ------------------------------------------------------------- PTX bits ----

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
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
// Barriers 1 and 2: one softmax warpgroup each.
__device__ __forceinline__ bool vote_group(int wg, bool any) {   // true where any of its threads asks
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)any), "r"(1 + wg)
        : "memory");
    return r != 0;
}
// Barrier 3: the decoding warps of V.
__device__ __forceinline__ bool vote_v(bool any) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 3, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)any)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_group(int wg) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + wg) : "memory"); }

// This warp's 32 TMEM lanes, N = 8 or 16 consecutive columns each.
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&v)[16]) { tc::tmem_ld16(t, v); }
__device__ __forceinline__ void tmem_ld(uint32_t t, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(t)
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(t),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] x B[smem]^T; issued by one thread.
__device__ __forceinline__ void mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

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

// A wait of the roles that run on after a failure: no waiting once *abort is
// set (they then arrive for work that was not done, but never on raw_empty, so
// that no copy is requested into a stage that another is still on its way to).
// One lane looks; a look at a phase that does not complete lasts kTreeLookNs
// (the hardware's suspension: 4.01 us measured), so the limit of the looks is one
// of time.  The warp waits for that lane.  Kept short: it stands in 20 places, and
// the roles' code has to stay in the instruction cache together (with the timer
// read in this loop the measured calls took 2 to 16 % longer, with a suspension of
// its own up to 10 %).
__device__ __forceinline__ bool wait_lane(uint64_t* bar, uint32_t parity, const Args& a, volatile int* abort,
                                          uint32_t looks = kTreeLooks) {
#pragma unroll 1
    for (uint32_t i = 0; i < looks; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    atomicOr(a.status, STATUS_TIMEOUT);
    return false;
}
// Copies or products in flight, after a failure.
__device__ __forceinline__ void wait_drained(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 0; i < kTreeLooks && !mbar_try_wait(bar, parity); ++i) {}
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Args& a, volatile int* abort) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0) ok = wait_lane(bar, parity, a, abort);
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}
// Whether a wait of the CTA has run out, the same in the whole warp.  A role
// that runs on arrives on its barriers without having waited, but only after it
// has seen *abort; so who finds it clear after a wait of its own was let
// through by work that was done.
__device__ __forceinline__ bool failed(volatile int* abort) { return __any_sync(0xffffffffu, *abort != 0); }

// Whether the unit's piece (m.piece[unit mod 8]) is there; false after a failure.
__device__ __forceinline__ bool piece_ready(Misc& m, uint32_t unit, const Args& a) {
    return wait_warp(&m.piece_full[unit & 7], (unit >> 3) & 1, a, &m.abort);
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

// Bits of the largest fp16 scale with which no code leaves fp16's range (65504
// over a power of two).
template <int T> __host__ __device__ constexpr uint32_t half_max_scale() { return 0x7BFFu - ((T == T_Q8_0 ? 7u : (T == T_Q5_0 ? 4u : 3u)) << 10); }

// One 32-block, read as words from a 2-byte aligned shared address.
template <int T> struct Block {
    static constexpr int W = Fmt<T>::BB / 4;   // words past the scale: 8, 4 or 5
    uint32_t w[W], d;                          // d: the scale's bits
    __device__ __forceinline__ explicit Block(const uint8_t* p) {
        const uint32_t at = smem_u32(p), odd = at & 2;   // the block starts 2 bytes into a word
        const uint8_t* q = p + 2 - (odd ^ 2);            // the word that holds the first byte past the scale
        uint32_t prev = hm::lds32(q);
        d = ld_u16(p);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const uint32_t next = hm::lds32(q + 4 * i + 4);
            w[i] = __funnelshift_r(prev, next, 8 * (odd ^ 2));
            prev = next;
        }
    }
    // Chunk k (0..3): code (exact) * d.
    __device__ __forceinline__ uint4 chunk(int k, uint32_t d2) const {
        using hm::and_or;
        using hm::and_xor;
        using hm::hadd2;
        const auto value = [d2](uint32_t code) { return hmul2(code, d2); };
        if constexpr (T == T_Q8_0) {   // 0x6480 ^ byte = 1152 + (signed byte)
            const uint32_t x = w[2 * k], y = w[2 * k + 1];
            return make_uint4(value(hadd2(and_xor(x, 0x00FF00FFu, 0x64806480u), 0xE480E480u)),
                              value(hadd2(and_xor(x >> 8, 0x00FF00FFu, 0x64806480u), 0xE480E480u)),
                              value(hadd2(and_xor(y, 0x00FF00FFu, 0x64806480u), 0xE480E480u)),
                              value(hadd2(and_xor(y >> 8, 0x00FF00FFu, 0x64806480u), 0xE480E480u)));
        } else if constexpr (T == T_Q4_0) {   // low nibbles 1024 + q - 1032, high ones 64 + q - 72
            const uint32_t x = w[k], y = x >> 8;
            return make_uint4(value(hadd2(and_or(x, 0x000F000Fu, 0x64006400u), 0xE408E408u)),
                              value(hadd2(and_or(y, 0x000F000Fu, 0x64006400u), 0xE408E408u)),
                              value(hadd2(and_or(x, 0x00F000F0u, 0x54005400u), 0xD480D480u)),
                              value(hadd2(and_or(y, 0x00F000F0u, 0x54005400u), 0xD480D480u)));
        } else {   // the fifth bits of 4 elements spread to bit 4 of their bytes; 1024 + q - 1040
            const uint32_t qh = w[0], x = w[1 + k];
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

// The warp's maxima of v[0 .. C) (NaN aside): lane l gets column l mod C in
// v[0], by exchanging halves.
template <int C>
__device__ __forceinline__ void warp_max_columns(float (&v)[C], int lane) {
#pragma unroll
    for (int o = 16; o >= C; o >>= 1)
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = fmaxf(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
#pragma unroll
    for (int o = C / 2; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool up = lane & o;
            const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
}

// One piece of a unit by a softmax warpgroup (wg 0, 1), which has C columns
// (rows; 8, 16 or 32): C wg .. C wg + C - 1.  tile: running count of the CTA's
// tiles; unit: of its pieces.  The columns are walked eight at a time in rolled
// loops: the roles share an instruction cache, and copies of this code for
// each C, unrolled, made every role's tile a third slower.
template <int T, int D>
__device__ __forceinline__ void softmax_piece(const Args& a, Misc& m, uint8_t* sp, uint32_t tmem, const Piece& p, uint32_t& tile,
                                              uint32_t unit, uint8_t* part, int wg, int C) {
    using G = Geo<T, D>;
    constexpr int CW = 8;
    const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, tid = 32 * wq + lane, c0 = C * wg;
    const uint32_t lanes = tmem + ((uint32_t)(32 * wq) << 16);
    const uint64_t* seen = m.seen[unit & 3] + c0;
    volatile int* abort = &m.abort;
    const int t0 = p.t0, t1 = p.t1, ctx = p.q.ctx;
    const float* mul = m.colc[unit & 3] + c0;
#pragma unroll 1
    for (int t = t0; t < t1; ++t, ++tile) {
        const uint32_t b = tile & 1;
        if (lane == 0) {
            wait_lane(&m.s_full[b], (tile >> 1) & 1, a, abort);
            if (tile >= 2) wait_lane(&m.pv_done[b], ((tile >> 1) - 1) & 1, a, abort);   // the P buffer is free
        }
        __syncwarp();
        tc::fence_after_sync();
        const int pos0 = t * G::BN;
        const uint4 vw = m.valid[0][tile & 15];
        const bool all = pos0 + G::BN <= ctx && (vw.x & vw.y) == 0xffffffffu && (G::BN == 64 || (vw.z & vw.w) == 0xffffffffu);
        const uint32_t mine = wq == 0 ? vw.x : wq == 1 ? vw.y : wq == 2 ? vw.z : vw.w;
        const bool here = (mine >> lane) & 1;   // the position exists (false past BN)
        const int j = pos0 + tid - ctx;         // drafted token at this position, if >= 0
        uint8_t* row = sp + b * G::PB + tid * 128;
        // CW scores from column h on.  A hidden score becomes the infinity
        // that the column's multiplier turns into -inf.  (No branch per
        // column: with them a tile with drafted positions took 10,000 clocks.)
        const uint32_t* seen_j = reinterpret_cast<const uint32_t*>(seen) + (j >= 32 ? 1 : 0);   // the half with bit j
        const uint32_t shift = j & 31, committed = j < 0, exists = here;
        auto load = [&](int h, uint32_t (&s)[CW]) {
            tmem_ld(lanes + 64 * b + c0 + h, s);
            tc::tmem_wait_ld();
            if (!all) {
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    const uint32_t vis = ((seen_j[2 * (h + c)] >> shift) | committed) & exists;
                    s[c] = vis ? s[c] : 0xff800000u ^ (__float_as_uint(mul[h + c]) & 0x80000000u);
                }
            }
        };
        // Once round for an ordinary tile; one whose scores outgrow the
        // references (x > kOver) gets new ones and comes round again, and so
        // does a unit's first tile.
        bool renew = t == t0;
#pragma unroll 1
        for (int round = 0;; ++round) {
            if (renew) {
#pragma unroll 1
                for (int h = 0; h < (G::BN == 128 || wq < 2 ? C : 0); h += CW) {
                    uint32_t s[CW];
                    float y[CW];
                    load(h, s);
#pragma unroll
                    for (int c = 0; c < CW; ++c) y[c] = __uint_as_float(s[c]) * mul[h + c];
                    warp_max_columns<CW>(y, lane);
                    if (lane < CW) m.wmax[wq][c0 + h + lane] = y[0];
                }
                sync_group(wg);
                if (tid < C) {
                    const int c = c0 + tid;
                    float top = fmaxf(m.wmax[0][c], m.wmax[1][c]);
                    if (G::BN == 128) top = fmaxf(top, fmaxf(m.wmax[2][c], m.wmax[3][c]));
                    const float old = t == t0 ? -INFINITY : m.ref[c], now = fmaxf(fmaxf(old, top), -INFINITY);   // never NaN
                    m.factor[c] = old == -INFINITY ? 0.0f : ex2(old - now);
                    m.ref[c] = now;
                    m.cmul[c] = mul[tid];
                    m.cref[c] = now == -INFINITY ? 1e30f : kLift - now;   // nothing visible yet: whatever comes outgrows it
                }
                sync_group(wg);
                if (t != t0) {   // the sums so far on the new references
                    wait_warp(&m.pv_done[b ^ 1], ((tile - 1) >> 1) & 1, a, abort);
                    tc::fence_after_sync();
                    // the rows' sums, O^T, the large blocks' O^T
                    const int sets = 1 + (*(volatile unsigned*)&m.used[unit & 7] ? 2 : 1) * (D == 256 ? 2 : 1);
#pragma unroll 1
                    for (int k = 0; k < sets; ++k) {
                        const uint32_t at = lanes + c0 + (k == 0 ? G::TL : D == 256 ? kTmemO + 32 * (k - 1) : kTmemO + 64 * (k - 1));
#pragma unroll 1
                        for (int h = 0; h < C; h += 8) {
                            uint32_t v[8];
                            tmem_ld(at + h, v);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 8; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * m.factor[c0 + h + c]);
                            tmem_st(at + h, v);
                        }
                    }
                    tmem_wait_st();
                }
            }
            // Scores to (lifted) probabilities, fp16, the position's row of P.
            float mx = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < (G::BN == 128 || wq < 2 ? C : 0); h += CW) {   // at d = 256 only 64 lanes are positions
                uint32_t s[CW], o[4];
                load(h, s);
                const float4* k4 = reinterpret_cast<const float4*>(&m.cmul[c0 + h]);
                const float4* r4 = reinterpret_cast<const float4*>(&m.cref[c0 + h]);
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 k = k4[i / 4], r = r4[i / 4];
                    const float2 u = unpair(fma2(pair(s[i], s[i + 1]), pair(k.x, k.y), pair(r.x, r.y)));
                    const float2 v = unpair(fma2(pair(s[i + 2], s[i + 3]), pair(k.z, k.w), pair(r.z, r.w)));
                    mx = fmaxf(fmaxf(mx, fmaxf(u.x, u.y)), fmaxf(v.x, v.y));
                    o[i / 2] = pack_f16(ex2(u.x), ex2(u.y));
                    o[i / 2 + 1] = pack_f16(ex2(v.x), ex2(v.y));
                }
                *reinterpret_cast<uint4*>(row + ((((c0 + h) / 8) ^ (tid & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (!vote_group(wg, mx > kOver) || round == 2) break;
            renew = true;
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_full[b]);   // and S^T has been read
    }
    // Epilogue.
    const bool whole = t0 == 0 && t1 == p.nt;
    float* po = reinterpret_cast<float*>(part);
    const uint32_t last = tile - 1;
    wait_warp(&m.pv_done[last & 1], (last >> 1) & 1, a, abort);
    tc::fence_after_sync();
    const unsigned used = *(volatile unsigned*)&m.used[unit & 7];
    const int64_t* rowoff = m.rowoff[unit & 3] + c0;
    const int rows = p.rows;
    // After a failure rowoff may never have been written: nothing is stored.
    const int halves = failed(abort) ? 0 : (D == 256 ? 2 : 1);
#pragma unroll 1
    for (int half = 0; half < halves; ++half) {
        const int blk = 4 * half + wq;
        if (blk >= G::NB) break;   // lanes past d (warp-uniform)
        const int e = 32 * blk + element_of<T>(lane);
        const uint64_t bad = m.bad_ctx[unit & 7][blk] ? ~uint64_t(0) : m.bad_draft[unit & 7][blk];
        const bool bad_all = m.bad_ctx[unit & 7][blk] != 0;
#pragma unroll 1
        for (int h = 0; h < C; h += 8) {
            uint32_t v[8], l[8];
            tmem_ld(lanes + kTmemO + 32 * half + c0 + h, v);
            tmem_ld(lanes + G::TL + c0 + h, l);   // every lane has the rows' sums
            tc::tmem_wait_ld();
            if (used) {
                uint32_t u[8];
                tmem_ld(lanes + kTmemBig + 32 * half + c0 + h, u);
                tc::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = __float_as_uint(fmaf(kBig, __uint_as_float(u[c]), __uint_as_float(v[c])));
            }
            if (bad) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (bad_all || (bad & seen[h + c])) v[c] = 0x7fffffffu;
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int col = c0 + h + c;
                const float o = __uint_as_float(v[c]), sum = __uint_as_float(l[c]);
                if (whole) {   // a row that saw nothing: zeros
                    const __nv_bfloat16 r = __float2bfloat16_rn(sum == 0.0f ? 0.0f : __fdividef(o, sum));
                    if (rowoff[h + c] >= 0) a.out[rowoff[h + c] + e] = r;
                } else {
                    if (col < rows) po[col * D + e] = o;
                    if (blk == 0 && lane == c) *reinterpret_cast<float2*>(po + kRows * D + 2 * col) = make_float2(m.ref[col], sum);
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) {
        mbar_arrive(&m.o_empty);
        mbar_arrive(&m.piece_free[unit & 7]);
    }
}

// --------------------------------------------------------------- kernel ----

template <int T, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const Args a) {
    using G = Geo<T, D>;
    extern __shared__ uint8_t smem_raw[];
    // Aligned by pointer arithmetic: through an integer the compiler would lose
    // the address space, and every shared access would be a generic one.
    uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
    uint8_t* sv = smem;                 // V tiles
    uint8_t* sq = sv + kV * G::VB;      // queries
    uint8_t* sp = sq + G::QB;           // P
    uint8_t* raw = sp + 2 * G::PB + 1024;   // packed tiles; before them eight rows of ones
    Misc& m = *reinterpret_cast<Misc*>(raw + G::NS * G::RAW);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &m.abort;

    pdl_launch_dependents();
    if (warp == 1) {
        tc::tmem_alloc(&m.tmem, kTmem);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < G::NS; ++i) {
            mbar_init(&m.raw_full[i], 1);
            mbar_init(&m.raw_empty[i], kDw);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m.k_full[i], kDw);
            mbar_init(&m.k_empty[i], 1);
            mbar_init(&m.v_full[i], kDw);
            mbar_init(&m.v_empty[i], 1);
            mbar_init(&m.s_full[i], 1);
            mbar_init(&m.p_full[i], 8);
            mbar_init(&m.pv_done[i], 1);
            mbar_init(&m.drain[i], 1);
        }
        mbar_init(&m.q_full, kDw);
        mbar_init(&m.q_empty, 1);
        mbar_init(&m.o_empty, 8);
        mbar_init(&m.big_full, kDw);
        mbar_init(&m.big_empty, 1);
        for (int i = 0; i < 8; ++i) {
            mbar_init(&m.piece_full[i], 1);
            mbar_init(&m.piece_free[i], 8);
        }
        m.abort = 0;
        fence_barrier_init();
    }
    if (tid >= 128 && tid < 192) *reinterpret_cast<uint4*>(raw - 1024 + 16 * (tid - 128)) = make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u);
    fence_proxy_async_smem();
    if (tid >= 64 && tid < 128) {
        m.bad_draft[(tid >> 3) & 7][tid & 7] = 0;
        m.bad_ctx[(tid >> 3) & 7][tid & 7] = 0;
    }
    // The list's length, then the request that holds this CTA's first tile:
    // running sums over the requests, kThreads of them at a time.
    int total = 0, per = 0, x0 = 0;
    {
        Req q{0, 0, 0, 0};
        int w = 0, upto = 0;   // this thread's request: its tiles, their end in the list
        auto sums = [&](int r0, int carry) {
            const int r = r0 + tid;
            q = r < a.n_req ? req_of(a, r) : Req{0, 0, 0, 0};
            w = work_of<G::BN, G::NR>(a, q);
            int v = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            __syncthreads();
            if (lane == 31) m.scan[warp] = v;
            __syncthreads();
            int s = lane < kThreads / 32 ? m.scan[lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += u;
            }
            upto = carry + v + (warp ? __shfl_sync(0xffffffffu, s, warp - 1) : 0);
            return carry + __shfl_sync(0xffffffffu, s, 31);
        };
        auto found = [&](int r0) {
            if (upto - w <= x0 && x0 < upto) {
                m.start_r = r0 + tid;
                m.start_base = upto - w;
                m.start_w = w;
                m.start_q = q;
            }
        };
#pragma unroll 1
        for (int r0 = 0; r0 < a.n_req; r0 += kThreads) total = sums(r0, total);
        per = (total + a.ctas - 1) / a.ctas;
        x0 = (int)blockIdx.x * per;
        if (a.n_req <= kThreads) {
            found(0);
        } else {
            int carry = 0;
#pragma unroll 1
            for (int r0 = 0; r0 < a.n_req; r0 += kThreads) {
                carry = sums(r0, carry);
                found(r0);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = m.tmem;
    const int x1 = min(x0 + per, total);
    // Registers per thread of the seven warpgroups: 104, 2 x 88, 2 x 48, 2 x 64, within the launch's 7 x 72.
    // (With fewer the copiers' loop spills, and a spill is a trip to L2: shared memory leaves no L1.)
    if (warp >= kSm && warp < kKd) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
        const int wg = (warp - kSm) >> 2;
        uint8_t* parts = a.ws + (int64_t)a.ctas * sizeof(Cut) + 2 * (int64_t)blockIdx.x * part_bytes<D>();
        uint32_t tile = 0, unit = 0;
#pragma unroll 1
        for (;; ++unit) {
            if (vote_group(wg, !piece_ready(m, unit, a))) break;
            const Piece& p = m.piece[unit & 7];
            const int rows = p.rows;
            if (rows == 0) break;
            uint8_t* part = parts + (p.t0 == 0 && p.u0 != x0 ? part_bytes<D>() : 0);
            softmax_piece<T, D>(a, m, sp, tmem, p, tile, unit, part, wg, cols_of(rows) / 2);
        }
    } else if (warp >= kKd && warp < kVd) {
        // K: a lane is a position; two warps per 32 positions share its items.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        uint32_t tile = 0;
        const int wq = warp & 3, pos = 32 * wq + lane, h = (warp - kKd) >> 2;
        const uint8_t* row0 = raw + pos * G::RB;
        const uint32_t to0 = tmem + ((uint32_t)(32 * wq) << 16) + kTmemK;
        uint32_t st = 0, rph = 0;   // the K tile's ring stage and its phase
#pragma unroll 1
        for (uint32_t unit = 0; piece_ready(m, unit, a) && m.piece[unit & 7].rows; ++unit) {
            const uint32_t end = tile + (m.piece[unit & 7].t1 - m.piece[unit & 7].t0);
#pragma unroll 1
            for (; tile < end; ++tile) {
                const uint32_t b = tile & 1;
                if (lane == 0) {
                    if (tile >= 2) wait_lane(&m.k_empty[b], ((tile >> 1) - 1) & 1, a, abort);
                    wait_lane(&m.raw_full[st], rph, a, abort);
                }
                __syncwarp();
                tc::fence_after_sync();
                if (32 * wq < G::BN) {
                    const uint8_t* row = row0 + st * G::RAW;
                    const uint32_t to = to0 + b * G::KC;
                    uint32_t top = 0;   // largest scale
#pragma unroll 1
                    for (int i = h; i < G::NB; i += 2) {
                        const Block<T> blk(row + i * Fmt<T>::BB);
                        const uint32_t d2 = hm::dup16(blk.d);
                        uint32_t v[16];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 u = blk.chunk(c, d2);
                            v[4 * c] = u.x, v[4 * c + 1] = u.y, v[4 * c + 2] = u.z, v[4 * c + 3] = u.w;
                        }
                        top = max(top, blk.d & 0x7fffu);
                        tmem_st(to + 16 * i, v);
                    }
                    tmem_wait_st();
                    // A value past fp16's range becomes NaN, and so does every score it enters: as an infinity it
                    // could make the score -inf, and the position would be left out in silence.
                    if (__any_sync(0xffffffffu, top > half_max_scale<T>())) {
#pragma unroll 1
                        for (int i = h; i < G::NB; i += 2) {
                            uint32_t v[16];
                            tmem_ld(to + 16 * i, v);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c) v[c] = hfma2(v[c], 0u, v[c]);   // inf * 0 is NaN, x * 0 + x is x
                            tmem_st(to + 16 * i, v);
                        }
                        tmem_wait_st();
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&m.k_full[b]);
                    if (!*abort) mbar_arrive(&m.raw_empty[st]);   // after a failure the copy may still be under way
                }
                if ((st += 2) == G::NS) st = 0, rph ^= 1;
            }
        }
    } else if (warp >= kVd) {
        // V: a warp's lanes are SPW positions by 32 / SPW items of the row, so
        // that its word loads fall into 32 different banks (a row's items are
        // 17, 9 or 11 words apart, odd; positions 1, 2 or 4 times that) and
        // eight neighbouring lanes' 16-byte stores into the eight bank groups
        // of swizzled rows.  Before a unit's first tile, its queries.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        constexpr int SPW = D <= 64 ? 32 : 2048 / D;
        static_assert(G::ITEMS <= kDw * 32, "an item per decoding thread");
        uint32_t tile = 0, unit = 0;
        const int dt = tid - 32 * kVd;
        const bool mine = dt < G::ITEMS;
        const int pos = mine ? (dt / 32) * SPW + lane % SPW : 0, seg = mine ? lane / SPW : 0;
        const uint8_t* src0 = raw + pos * G::RB + seg * 2 * Fmt<T>::BB;
        uint8_t* line0 = sv + seg * G::CHB + pos * 128;
        uint32_t st = 1, rph = 0;   // the V tile's ring stage and its phase
        uint32_t bigs = 0;          // tiles with large blocks so far
#pragma unroll 1
        for (;; ++unit) {
            if (vote_v(!piece_ready(m, unit, a))) break;
            const Piece& p = m.piece[unit & 7];
            if (p.rows == 0) break;
            {
                // The queries, a thread per 32 elements, to fp16 times a power of
                // two that brings the row's largest magnitude to 2^14 .. 2^15
                // (bf16's 8 bits are exact).
                constexpr int TPR = D / 32;   // threads per row
                static_assert(G::NR * TPR <= kDw * 32, "a thread per query block");
                const int rows = p.rows, row = dt / TPR, sub = dt % TPR, N = cols_of(rows), tok = token_of(a, p.row0 + row);
                const int head = p.g * a.G + p.row0 + row - tok * a.G;
                const bool live = row < rows;
                uint32_t x[16];   // pairs of elements
                uint64_t seen = 0;
                if (live) {
                    const uint4* q = reinterpret_cast<const uint4*>(a.q + (p.q.tok0 + tok) * a.q_stride + head * D + 32 * sub);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 u = q[c];
                        x[4 * c] = u.x, x[4 * c + 1] = u.y, x[4 * c + 2] = u.z, x[4 * c + 3] = u.w;
                    }
                    if (sub == 0) seen = seen_of(a, p.q, tok);
                } else {
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = 0;
                }
                uint32_t top = 0;   // largest magnitude, as bf16 bits
#pragma unroll
                for (int c = 0; c < 16; ++c) top = __vmaxu2(top, x[c] & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
#pragma unroll
                for (int o = 1; o < TPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                int ex = (int)(top >> 7) - 127 - 14;   // the largest magnitude is below 2^(ex + 15)
                if (top == 0 || ex > 113) ex = 0;      // nothing, or not finite
                ex = max(ex, -126);                    // the factors stay normal
                const float down = __uint_as_float((uint32_t)(127 - ex) << 23), up = __uint_as_float((uint32_t)(127 + ex) << 23);
                // The scores' multiplier.  Two kinds of row get a multiplier of 1, which turns a hidden score's infinity
                // into -inf, and queries that give the visible scores: NaN where the query or the multiplier is not finite
                // (all of them infinite with one sign would be a softmax of nothing), 0 where the multiplier is 0 (the
                // scale is, or the product underflows).
                float mul = a.scale * 1.44269504088896341f * up;
                const bool no_score = top >= 0x7f80u || !(fabsf(mul) <= 3.402823466e38f);
                if (no_score || mul == 0.0f) {
                    mul = 1.0f;
#pragma unroll
                    for (int c = 0; c < 16; ++c) x[c] = no_score ? 0x7fff7fffu : 0u;
                }
                if (unit > 0) wait_warp(&m.q_empty, (unit - 1) & 1, a, abort);
                if (row < N) {
                    uint8_t* to = sq + (sub >> 1) * (G::NR * 128) + row * 128;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {   // element_of's order: 0, 2, 1, 3 of each four
                        const int i = T == T_Q8_0 ? 4 * k : 2 * k, j = T == T_Q8_0 ? 4 * k + 2 : 8 + 2 * k;
                        uint32_t o[4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t u = x[h ? j : i], v = x[(h ? j : i) + 1];
                            o[2 * h] = pack_f16(__uint_as_float(u << 16) * down, __uint_as_float(v << 16) * down);
                            o[2 * h + 1] = pack_f16(__uint_as_float(u & 0xffff0000u) * down, __uint_as_float(v & 0xffff0000u) * down);
                        }
                        *reinterpret_cast<uint4*>(to + ((((sub & 1) * 4 + k) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    if (sub == 0) {
                        m.colc[unit & 3][row] = mul;
                        m.seen[unit & 3][row] = seen;
                        m.rowoff[unit & 3][row] = live ? (p.q.tok0 + tok) * a.out_stride + head * D : -1;
                    }
                }
                // The flags of unit + 1 (last of unit - 7, long done) start clear;
                // no warp reaches that unit's V before q_full.
                if (dt < 8) {
                    m.bad_draft[(unit + 1) & 7][dt] = 0;
                    m.bad_ctx[(unit + 1) & 7][dt] = 0;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.q_full);
            }
            int j = p.t0 * G::BN + pos - p.q.ctx;   // drafted token at the thread's position, if >= 0
            const uint32_t end = tile + (p.t1 - p.t0);
#pragma unroll 1
            for (; tile < end; ++tile, j += G::BN) {
                const uint32_t b = tile & 1;
                if (lane == 0) {
                    if (tile >= 2) wait_lane(&m.v_empty[b], ((tile >> 1) - 1) & 1, a, abort);
                    wait_lane(&m.raw_full[st], rph, a, abort, a.looks);
                }
                __syncwarp();
                const bool valid = mine && ((reinterpret_cast<const uint32_t*>(&m.valid[1][tile & 15])[pos >> 5] >> (pos & 31)) & 1);
                const uint8_t* src = src0 + st * G::RAW;
                // Blocks whose scale is finite but too large for fp16 times a code are large ones, those whose scale is
                // not finite are recorded; both are zeros in the tile.
                bool big = false;
                uint32_t good = 0;   // bit per block
#pragma unroll
                for (int i = 0; i < G::ITEM / 32; ++i) {
                    const float d = fabsf(h2f(ld_u16(src + i * Fmt<T>::BB)));
                    if (valid) good |= 1u << i;
                    if (valid && !(d * code_max<T>() <= 65504.0f)) {
                        good ^= 1u << i;
                        big = big || d <= 65504.0f;
                        if (!(d <= 65504.0f)) {
                            const int blk = 2 * seg + i;
                            if (j < 0) atomicOr(&m.bad_ctx[unit & 7][blk], 1u);
                            else atomicOr(&m.bad_draft[unit & 7][blk], 1ull << (j & 63));
                        }
                    }
                }
                big = vote_v(big);
                if (dt == 0) m.big_tile[tile & 15] = big;
                uint8_t* line = line0 + b * G::VB;
                auto blocks = [&](uint32_t which, uint32_t times) {   // the others are zeros; times: the scales' factor, two halves
#pragma unroll 1
                    for (int i = 0; i < G::ITEM / 32; ++i) {
                        const Block<T> blk(src + i * Fmt<T>::BB);
                        const uint32_t d2 = times == 0x3C003C00u ? hm::dup16(blk.d) : hmul2(hm::dup16(blk.d), times);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint4 o = blk.chunk(c, d2);
                            if (!((which >> i) & 1)) o = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(line + (((4 * i + c) ^ (pos & 7)) << 4)) = o;
                        }
                    }
                };
                if (mine) blocks(good, 0x3C003C00u);   // 1
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.v_full[b]);
                if (big) {   // then the large blocks, in the same buffer once its product is done
                    if (lane == 0) wait_lane(&m.v_empty[b], (tile >> 1) & 1, a, abort);
                    __syncwarp();
                    uint32_t large = 0;
#pragma unroll
                    for (int i = 0; i < G::ITEM / 32; ++i) {
                        const float d = fabsf(h2f(ld_u16(src + i * Fmt<T>::BB)));
                        if (valid && d * code_max<T>() > 65504.0f && d <= 65504.0f) large |= 1u << i;
                    }
                    if (mine) blocks(large, 0x20002000u);   // 2^-7 (exact: a large scale is above 2^8)
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&m.big_full);
                        wait_lane(&m.big_empty, bigs & 1, a, abort);
                    }
                    __syncwarp();
                    ++bigs;
                }
                if (lane == 0 && !*abort) mbar_arrive(&m.raw_empty[st]);
                if ((st += 2) == G::NS + 1) st = 1, rph ^= 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        if (warp == 0 || warp == 3) {
            // Copies: the tile's rows of every page it touches, K's by warp 0
            // (which also walks the list and publishes the pieces), V's by warp 3.
            const int kv = warp == 3;
            const uint8_t* pool = kv ? a.V : a.K;
            uint32_t tile = 0, st = kv, rph = 1;   // ring stage; phase of its release (the first round passes at once)
            const uint64_t pol = policy_evict_first();
            bool ok = true;
            const int pl = a.pool.page_log2, sl = min(pl, G::BN == 64 ? 6 : 7);   // log2 of a slab's positions
            const int span = 1 << sl, slabs = G::BN >> sl;
            const int64_t page_bytes = ((int64_t)a.pool.n_kv << pl) * G::RB;
            const bool leader = tc::elect_one();
            Walk<G::BN, G::NR> w{x0, x1, m.start_base, m.start_w, m.start_r, m.start_q};
#pragma unroll 1
            for (uint32_t unit = 0; ok; ++unit) {
                Piece p;
                if (kv) {
                    ok = piece_ready(m, unit, a);
                    if (!ok) break;
                    p = m.piece[unit & 7];
                } else {
                    const bool more = w.next(a, p);
                    if (unit >= 8 && (!wait_warp(&m.piece_free[unit & 7], ((unit >> 3) - 1) & 1, a, abort) || failed(abort))) { ok = false; break; }
                    if (!more) p.rows = 0;
                    if (lane == 0) {
                        m.piece[unit & 7] = p;
                        mbar_arrive(&m.piece_full[unit & 7]);
                    }
                    if (unit == 0) {   // a unit cut at this CTA's start, for join_kernel
                        Cut c{};
                        if (more && p.t0 > 0 && p.u0 / per == (int)blockIdx.x - 1) {
                            c.rows = p.rows;
                            c.first = (int)blockIdx.x - 1;
                            c.last = (p.u0 + p.nt - 1) / per;
                            c.first_slot = 2 * c.first + (p.u0 != c.first * per);
                            c.tok0 = p.q.tok0;
                            c.row0 = p.row0;
                            c.g = p.g;
                        }
                        if (lane == 0) reinterpret_cast<Cut*>(a.ws)[blockIdx.x] = c;
                    }
                }
                if (p.rows == 0) break;
                const int len = p.q.len;
                const bool held = kv && a.hold - tile < (uint32_t)(p.t1 - p.t0);   // the copies stop inside the unit
                const int t1 = held ? p.t0 + (int)(a.hold - tile) : p.t1;
                const bool shared = groups_of(p.q, a.G, G::NR) > 1;   // other row groups read these bytes too
                const int32_t* tab = a.table + (int64_t)p.r * a.table_stride;
                const uint8_t* head = pool + ((int64_t)p.g << pl) * G::RB;
                int pos = p.t0 * G::BN + lane * span;   // this lane's slab
                // Its page id, one tile ahead of the use.
                auto page_id = [&](int at) { return lane < slabs && at < len ? tab[at >> pl] : -1; };
                int ahead = page_id(pos);
#pragma unroll 1
                for (int t = p.t0; t < t1; ++t, ++tile, pos += G::BN) {
                    int id = ahead;
                    ahead = t + 1 < t1 ? page_id(pos + G::BN) : -1;
                    const bool live = lane < slabs && pos < len;
                    if (live && (id < 0 || id >= a.pool.n_pages)) {
                        atomicOr(a.status, STATUS_BAD_PAGE);
                        id = -1;
                    }
                    const int rows = id >= 0 && live ? min(span, len - pos) : 0;
                    const uint32_t bytes = (uint32_t)(rows * G::RB + 15) & ~15u;   // whole slabs are multiples of 16
                    uint32_t sum = G::BN * G::RB;
                    uint4 valid = make_uint4(~0u, ~0u, G::BN == 64 ? 0 : ~0u, G::BN == 64 ? 0 : ~0u);
                    if (__any_sync(0xffffffffu, lane < slabs && rows < span)) {   // not whole
                        sum = __reduce_add_sync(0xffffffffu, bytes);
                        // Lane L reports positions 4 L .. 4 L + 3, which lie in one slab.
                        const int left = __shfl_sync(0xffffffffu, rows, (4 * lane) >> sl) - ((4 * lane) & (span - 1));
                        uint32_t bits = 4 * lane < G::BN ? (left >= 4 ? 15u : left > 0 ? (1u << left) - 1 : 0u) : 0u;
                        bits <<= 4 * (lane & 7);
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
                        valid = make_uint4(__shfl_sync(0xffffffffu, bits, 0), __shfl_sync(0xffffffffu, bits, 8),
                                           __shfl_sync(0xffffffffu, bits, 16), __shfl_sync(0xffffffffu, bits, 24));
                    }
                    const uint32_t src_in = (pos & ((1 << pl) - 1)) * G::RB;   // inside the page's head
                    int good = 1;
                    if (lane == 0) {
                        good = wait_lane(&m.raw_empty[st], rph, a, abort);
                        m.valid[kv][tile & 15] = valid;   // published by the arrival
                        if (good) mbar_arrive_expect_tx(&m.raw_full[st], sum);
                    }
                    ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                    if (!ok) break;
                    // One lane issues: with an issuing lane per slab the copies take several hundred clocks each.
#pragma unroll 1
                    for (int i = 0; i < slabs; ++i) {
                        const uint32_t n = __shfl_sync(0xffffffffu, bytes, i);
                        const int64_t off = __shfl_sync(0xffffffffu, id, i) * page_bytes + __shfl_sync(0xffffffffu, src_in, i);
                        if (leader && n) {
                            uint8_t* dst = raw + st * G::RAW + i * span * G::RB;
                            if (shared) bulk_g2s_keep(dst, head + off, n, &m.raw_full[st]);
                            else bulk_g2s(dst, head + off, n, &m.raw_full[st], pol);
                        }
                    }
                    __syncwarp();
                    if ((st += 2) >= G::NS) st = kv, rph ^= 1;
                }
                if (held) break;
            }
            // Copies in flight land before the CTA may leave: the last phase of each stage (of one that was never used, the
            // phase before its first).
            if (failed(abort))
#pragma unroll 1
                for (uint32_t s = kv; s < G::NS; s += 2) wait_drained(&m.raw_full[s], rph ^ (s < st));
        } else if (warp == 1) {
            // Q K: the warp walks together, one lane issues.
            uint32_t tile = 0, unit = 0;
            bool ok = true;
            const bool leader = tc::elect_one();
            const uint64_t dq = tc::sdesc_k128(smem_u32(sq));
            for (; ok && (ok = piece_ready(m, unit, a)) && m.piece[unit & 7].rows; ++unit) {
                const Piece& p = m.piece[unit & 7];
                const uint32_t id = idesc_f16(cols_of(p.rows), false), begin = tile, end = tile + (p.t1 - p.t0);
#pragma unroll 1
                for (; tile < end; ++tile) {
                    const uint32_t b = tile & 1;
                    int good = 1;
                    if (lane == 0) {
                        if (tile == begin) good = wait_lane(&m.q_full, unit & 1, a, abort);
                        good = good && (tile < 2 || wait_lane(&m.p_full[b], ((tile >> 1) - 1) & 1, a, abort));   // S^T has been read
                        good = good && wait_lane(&m.k_full[b], (tile >> 1) & 1, a, abort);
                    }
                    ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                    if (!ok) break;
                    tc::fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_ta(tmem + 64 * b, tmem + kTmemK + b * G::KC + 8 * k, dq + ((k >> 2) * (G::NR * 8) + 2 * (k & 3)), id, k > 0);
                        tc::commit(&m.s_full[b]);
                        tc::commit(&m.k_empty[b]);
                        if (tile == end - 1) tc::commit(&m.q_empty);
                    }
                    __syncwarp();
                }
            }
            if (failed(abort)) {   // let the products in flight end
                if (leader) tc::commit(&m.drain[0]);
                __syncwarp();
                if (lane == 0) wait_drained(&m.drain[0], 0);
                __syncwarp();
            }
        } else {
            // P V.
            uint32_t tile = 0, unit = 0, bigs = 0;   // bigs: tiles with large blocks so far
            bool ok = true;
            const bool leader = tc::elect_one();
            // d <= 64: one chunk only, read twice (rows 64 .. 127 of O^T are not used)
            const uint64_t dv = sdesc_mn128(smem_u32(sv), D <= 64 ? 0 : G::CHB), dp = sdesc_mn128(smem_u32(sp), 0);
            // the rows' sums: a tile of ones in V's place (one 8-row atom, its row stride 0)
            const uint64_t ones = tc::sdesc_k128(smem_u32(sp + 2 * G::PB)) & ~(uint64_t(0x3FFF) << 32);
            for (; ok && (ok = piece_ready(m, unit, a)) && m.piece[unit & 7].rows; ++unit) {
                const Piece& p = m.piece[unit & 7];
                const uint32_t id = idesc_f16(cols_of(p.rows), true), id1 = id & ~(1u << 15), begin = tile, end = tile + (p.t1 - p.t0);
                bool used = false;   // large blocks
#pragma unroll 1
                for (; tile < end; ++tile) {
                    const uint32_t b = tile & 1;
                    int good = 1;
                    if (lane == 0) {
                        if (tile == begin && unit > 0) good = wait_lane(&m.o_empty, (unit - 1) & 1, a, abort);
                        good = good && wait_lane(&m.v_full[b], (tile >> 1) & 1, a, abort) &&
                               wait_lane(&m.p_full[b], (tile >> 1) & 1, a, abort);
                    }
                    ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                    if (!ok) break;
                    tc::fence_after_sync();
                    const bool big = *(volatile unsigned*)&m.big_tile[tile & 15] != 0;
                    const uint64_t da = dv + (uint64_t)(b * (G::VB >> 4)), db = dp + (uint64_t)(b * (G::PB >> 4));
                    if (leader) {
                        *(volatile unsigned*)&m.used[unit & 7] = used || big;
#pragma unroll
                        for (int half = 0; half < (D == 256 ? 2 : 1); ++half)
#pragma unroll
                            for (int k = 0; k < G::BN / 16; ++k)
                                tc::mma_bf16(tmem + kTmemO + 32 * half, da + (half * (G::CHB >> 3) + 128 * k), db + 128 * k, id, tile > begin || k > 0);
                        tc::commit(&m.v_empty[b]);
#pragma unroll
                        for (int k = 0; k < G::BN / 16; ++k)
                            tc::mma_bf16(tmem + G::TL, ones, db + 128 * k, id1, tile > begin || k > 0);
                    }
                    if (big) {   // the same in the whole warp
                        if (lane == 0) good = wait_lane(&m.big_full, bigs & 1, a, abort);
                        ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                        if (!ok) break;
                        tc::fence_after_sync();
                        if (leader) {
#pragma unroll 1
                            for (int i = 0; i < (D == 256 ? 2 : 1) * (G::BN / 16); ++i) {
                                const int half = i / (G::BN / 16), k = i % (G::BN / 16);
                                tc::mma_bf16(tmem + kTmemBig + 32 * half, da + (half * (G::CHB >> 3) + 128 * k), db + 128 * k, id, used || k > 0);
                            }
                            tc::commit(&m.big_empty);
                        }
                        used = true;
                        ++bigs;
                    }
                    if (leader) tc::commit(&m.pv_done[b]);
                    __syncwarp();
                }
            }
            if (failed(abort)) {
                if (leader) tc::commit(&m.drain[1]);
                __syncwarp();
                if (lane == 0) wait_drained(&m.drain[1], 0);
                __syncwarp();
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
// gridDim.y, ... (one per warp) of the unit cut at CTA c's start.  Launched for
// every call, also one without a cut unit; d = 256 spills 36 bytes of stores and
// 44 of loads a thread.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Args a) {
    constexpr int E = D / 32;
    pdl_wait_prior();
    const Cut c = reinterpret_cast<const Cut*>(a.ws)[blockIdx.x];
    const uint8_t* parts = a.ws + (int64_t)a.ctas * sizeof(Cut);
    constexpr int64_t PART = part_bytes<D>();
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
#pragma unroll 8
            for (int i = 0; i < min(32, n - i0); ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                sum += __shfl_sync(0xffffffffu, lf, i);
                const float* po = part(i0 + i) + row * D + lane;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += fi * po[32 * e];
            }
        }
        const int rr = c.row0 + row, tok = token_of(a, rr);
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

// Tiles of the largest call of this shape.
double attn_tree_max_tiles(int64_t n_req, int max_q, int64_t max_pos, int n_heads, int n_kv, int d) {
    const int bn = d == 256 ? 64 : 128, nr = d == 256 ? 32 : 64;
    return (double)n_req * n_kv * (((int64_t)max_q * (n_heads / n_kv) + nr - 1) / nr) * std::max<int64_t>(1, (max_pos + bn - 1) / bn);
}

// The grid: one CTA per SM, fewer when the call cannot have that many tiles.
static int tree_ctas(int64_t n_req, int max_q, int64_t max_pos, int n_heads, int n_kv, int d, int sms) {
    const double tiles = attn_tree_max_tiles(n_req, max_q, max_pos, n_heads, n_kv, d);
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
                             unsigned* status, uint32_t looks, uint32_t hold, int sms, cudaStream_t s) {
    const tree::Args a{static_cast<const __nv_bfloat16*>(q), n_tok, q_stride, K, V, Pool{n_pages, page_log2, n_kv, row_bytes},
                       table, table_stride, ctx, cu, mask, (int)n_req, max_q, n_heads / n_kv,
                       (uint32_t)(((1 << 19) + n_heads / n_kv - 1) / (n_heads / n_kv)), scale,
                       static_cast<__nv_bfloat16*>(out), out_stride, static_cast<uint8_t*>(ws),
                       tree_ctas(n_req, max_q, table_stride << page_log2, n_heads, n_kv, d, sms), status, looks, hold};
    switch (type) {
    case T_Q8_0: return tree::launch_d<T_Q8_0>(a, d, s);
    case T_Q5_0: return tree::launch_d<T_Q5_0>(a, d, s);
    case T_Q4_0: return tree::launch_d<T_Q4_0>(a, d, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace qk
