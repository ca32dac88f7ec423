// qk_kv.cu -- the paged KV cache's bookkeeping and its writers: page planning
// (block tables and slot maps from request lengths), rows quantized into
// their slots, and the move of a drafted tree's accepted rows.
#include <algorithm>

#include "qk_internal.h"
#include "qk_paged.cuh"
#include "qk_ptx.cuh"
#include "qk_qlanes.cuh"

namespace qk {
namespace kv {

// ------------------------------------------------------------- planning --
// Per request: grow = max(0, P_new - P_old), shrink = max(0, P_old - P_new),
// tokens = max(0, want - start); an invalid request has none of them.  Three
// running sums over the requests give everything else by index arithmetic:
//   the freed pages form one list (request order), which continues the stack
//   of n_free pages; page k of the growing requests, in order, is entry
//   avail - 1 - k of that joined list (avail = n_free + freed pages);
//   token i belongs to the request whose token sum brackets i.
// Every CTA computes the sums for itself (a few thousand integers from L2)
// and then takes its share of the requests' tables and of the tokens, so the
// call is one launch without a grid barrier.  That is safe because reads and
// writes are disjoint: stack entries below n_free and table entries below
// P_old are read, stack entries from n_free up and table entries from P_old
// up are written.  Latency bounds it: 4.0 us for 5 requests, 9.6 us for 997
// requests and 180,248 tokens (3.2 MB) with 1,024 tokens a CTA; with 4,096 a
// CTA it took 12.7 us.
constexpr int kPlanThreads = 1024;
constexpr int kTokensPerCta = 1024;

struct PlanArgs {
    const int32_t *have, *start, *want;
    int n_req, page_log2;
    int32_t* table;
    int64_t table_stride;
    int32_t* free_pages;
    int64_t free_cap;
    const int32_t* n_free;
    int32_t *n_free_out, *granted, *cu;
    int64_t* slots;
    int32_t *pos, *req;
    int64_t cap;
};

struct Change {
    int p_old, p_new, tokens;
    bool valid;
    __device__ __forceinline__ int grow() const { return max(0, p_new - p_old); }
    __device__ __forceinline__ int shrink() const { return max(0, p_old - p_new); }
};
__device__ __forceinline__ Change change_of(const PlanArgs& a, int r) {
    Change c{0, 0, 0, false};
    const int64_t h = a.have[r], w = a.want[r], s = a.start[r], m = (int64_t(1) << a.page_log2) - 1;
    const int64_t po = (h + m) >> a.page_log2, pn = (w + m) >> a.page_log2;
    if (h >= 0 && w >= 0 && s >= 0 && po <= a.table_stride && pn <= a.table_stride) {
        c.p_old = (int)po;
        c.p_new = (int)pn;
        c.tokens = (int)max((int64_t)0, w - s);
        c.valid = true;
    }
    return c;
}

__device__ __forceinline__ int sat32(int64_t v) { return (int)min(v, (int64_t)0x7fffffff); }

// First i in [lo, n] with sum[i] > v, less one: the bracket of v in a
// non-decreasing sum with sum[0] = 0.
__device__ __forceinline__ int bracket(const int* sum, int n, int v) {
    int lo = 0, hi = n;   // sum[lo] <= v; the answer is in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sum[mid] <= v) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
    extern __shared__ int sums[];   // grow, shrink, tokens: n_req + 1 each
    __shared__ int64_t warp_sum[3][32], carry[3];
    const int n = a.n_req, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* sg = sums;
    int* ss = sums + n + 1;
    int* st = sums + 2 * (n + 1);
    if (tid < 3) carry[tid] = 0;
    if (tid == 0) sg[0] = ss[0] = st[0] = 0;
    __syncthreads();
    for (int r0 = 0; r0 < n; r0 += kPlanThreads) {
        const int r = r0 + tid;
        int64_t v[3] = {0, 0, 0};
        if (r < n) {
            const Change c = change_of(a, r);
            v[0] = c.grow();
            v[1] = c.shrink();
            v[2] = c.tokens;
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t t = __shfl_up_sync(0xffffffffu, v[k], o);
                if (lane >= o) v[k] += t;
            }
        if (lane == 31)
#pragma unroll
            for (int k = 0; k < 3; ++k) warp_sum[k][warp] = v[k];
        __syncthreads();
        if (warp < 3) {
            int64_t w = warp_sum[warp][lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t t = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += t;
            }
            warp_sum[warp][lane] = w;   // inclusive over the warps
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int64_t total = carry[k] + (warp ? warp_sum[k][warp - 1] : 0) + v[k];
            if (r < n) (k == 0 ? sg : k == 1 ? ss : st)[r + 1] = sat32(total);
        }
        __syncthreads();
        if (tid < 3) carry[tid] += warp_sum[tid][31];
        __syncthreads();
    }
    const int n_free = (int)min(max((int64_t)*a.n_free, (int64_t)0), a.free_cap);
    const int freed = ss[n];
    const int64_t avail = (int64_t)n_free + freed;
    const int taken = sg[bracket(sg, n, sat32(avail))];   // the largest running sum that fits
    // Entry v of the joined list: a free page, or freed page v - n_free, an
    // old table entry of a shrinking request.
    auto entry = [&](int64_t v) -> int {
        if (v < n_free) return a.free_pages[v];
        const int f = (int)(v - n_free);
        const int r = bracket(ss, n, f);   // ss[r] <= f < ss[r + 1]
        const int64_t p_new = ((int64_t)a.want[r] + (1 << a.page_log2) - 1) >> a.page_log2;
        return a.table[r * a.table_stride + p_new + (f - ss[r])];
    };
    // Requests: tables, grants, token sums.
    const int gw = blockIdx.x * (kPlanThreads / 32) + warp, nw = gridDim.x * (kPlanThreads / 32);
    for (int r = gw; r < n; r += nw) {
        const Change c = change_of(a, r);
        const bool ok = c.valid && (c.grow() == 0 || sg[r + 1] <= avail);
        if (lane == 0) {
            a.granted[r] = ok;
            a.cu[r + 1] = st[r + 1];
        }
        if (ok)
            for (int k = lane; k < c.grow(); k += 32)
                a.table[r * a.table_stride + c.p_old + k] = entry(avail - 1 - (sg[r] + k));
    }
    const int64_t gt = (int64_t)blockIdx.x * kPlanThreads + tid, nt = (int64_t)gridDim.x * kPlanThreads;
    if (gt == 0) {
        a.cu[0] = 0;
        *a.n_free_out = sat32(avail - taken);
    }
    // Freed pages that no request took go onto the stack.
    for (int64_t i = gt; i < (int64_t)freed - taken; i += nt)
        if (n_free + i < a.free_cap) a.free_pages[n_free + i] = entry(n_free + i);
    // Tokens.
    const int total = st[n];
    for (int64_t i = gt; i < a.cap; i += nt) {
        int64_t slot = -1;
        int pos = -1, r = -1;
        if (i < total) {
            r = bracket(st, n, (int)i);
            pos = a.start[r] + ((int)i - st[r]);
            const int grow = sg[r + 1] - sg[r];
            if (grow == 0 || sg[r + 1] <= avail) {
                const int pi = pos >> a.page_log2;
                const int p_old = (int)(((int64_t)a.have[r] + (1 << a.page_log2) - 1) >> a.page_log2);
                const int id = pi < p_old ? a.table[r * a.table_stride + pi] : entry(avail - 1 - (sg[r] + pi - p_old));
                slot = ((int64_t)id << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
            }
        }
        a.slots[i] = slot;
        if (a.pos) a.pos[i] = pos;
        if (a.req) a.req[i] = r;
    }
}

// --------------------------------------------------------------- append --
// Four lanes share a 32-element block: lane e of the four holds elements
// 8 e .. 8 e + 7 (one 16-byte load of bf16, two of fp32, so a warp's loads
// are contiguous), the block's maximum is two shuffles, and each lane rounds
// its own eight codes with the quantizer's arithmetic (group_codes: the
// IEEE division's rounding).  A thread does its block of K and of V: the slot
// and the indexes serve both and both loads are in flight together.
// The bytes of the rows read and the blocks written are its floor, instructions
// bind it: 32,764 tokens of 8 heads of 128, bf16 to Q4_0 (153 MB), 73 us, 31 % of
// the measured copy rate, with 81 % of the issue slots used and DRAM at 24 % (its
// counters); 13 tokens 2.5 us.
// Staging the blocks in shared memory to store whole rows took 101 us, so the
// scattered stores are not what binds it.
constexpr int kAppendThreads = 256;

struct AppendArgs {
    const void *k, *v;
    int64_t n_tok, k_stride, v_stride;
    const int64_t* slots;
    uint8_t *K, *V;
    Pool pool;
    int nb;             // 32-blocks per (token, head)
    int64_t n_blocks;   // n_tok * n_kv * nb, of one pool
    bool k_vec, v_vec;  // 16-byte aligned rows
    unsigned* status;
};

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t at, bool vec, float (&x)[8]) {
    if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        uint32_t w[4];
        if (vec) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float* p = static_cast<const float*>(base) + at;
        if (vec) {
            const float4 f = __ldcs(reinterpret_cast<const float4*>(p)), g = __ldcs(reinterpret_cast<const float4*>(p + 4));
            x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w, x[4] = g.x, x[5] = g.y, x[6] = g.z, x[7] = g.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = p[i];
        }
    }
}

// The lane's part of one block, e of four, at dst (nullptr: nothing is written).
template <int T>
__device__ __forceinline__ void append_block(const float (&x)[8], uint8_t* dst, int e) {
    constexpr int kOff = T == T_Q8_0 ? 0 : (T == T_Q5_0 ? 16 : 8);
    constexpr int kLo = T == T_Q8_0 ? -128 : -kOff;
    constexpr int kHi = T == T_Q8_0 ? 127 : kOff - 1;
    constexpr float kDiv = T == T_Q8_0 ? 127.0f : (T == T_Q5_0 ? 15.0f : 7.0f);
    float m = 0.0f;   // NaN elements are skipped, as the quantizer's scan does
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t db = ql::half_bits(__fdiv_rn(m, kDiv));
    const float d = ql::half_val(db);
    uint32_t q[8];
    if (d > 0.0f) {
        group_codes<8, kLo, kHi, kOff>(x, d, q);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = (uint32_t)kOff;
    }
    const uint32_t w0 = ql::bytes4(q), w1 = ql::bytes4(q + 4);
    if constexpr (T == T_Q8_0) {
        if (dst) {
            if (e == 0) ql::st_u16(dst, db);
            uint8_t* p = dst + 2 + 8 * e;
            ql::st_u16(p, w0 & 0xffffu);
            ql::st_u16(p + 2, w0 >> 16);
            ql::st_u16(p + 4, w1 & 0xffffu);
            ql::st_u16(p + 6, w1 >> 16);
        }
    } else {
        // Byte j holds element j (low nibble) and j + 16 (high): lanes 0 and
        // 1 take the high nibbles from lanes 2 and 3.
        const uint32_t h0 = __shfl_xor_sync(0xffffffffu, w0, 2), h1 = __shfl_xor_sync(0xffffffffu, w1, 2);
        uint32_t fifth = 0;
        if constexpr (T == T_Q5_0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) fifth |= ((q[i] >> 4) & 1u) << i;   // byte e of the fifth-bit word
        }
        if (dst) {
            uint8_t* qs = dst + (T == T_Q5_0 ? 6 : 2);
            if (e == 0) ql::st_u16(dst, db);
            if (T == T_Q5_0) dst[2 + e] = (uint8_t)fifth;
            if (e < 2) {
                const uint32_t n0 = (w0 & 0x0F0F0F0Fu) | ((h0 & 0x0F0F0F0Fu) << 4);
                const uint32_t n1 = (w1 & 0x0F0F0F0Fu) | ((h1 & 0x0F0F0F0Fu) << 4);
                uint8_t* p = qs + 8 * e;
                ql::st_u16(p, n0 & 0xffffu);
                ql::st_u16(p + 2, n0 >> 16);
                ql::st_u16(p + 4, n1 & 0xffffu);
                ql::st_u16(p + 6, n1 >> 16);
            }
        }
    }
}

template <int T, bool BF16>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    const int64_t b = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) >> 2;   // block of K and of V
    const int e = threadIdx.x & 3;
    const bool live = b < a.n_blocks;
    const int per_tok = a.pool.n_kv * a.nb;
    // 32-bit divisions where the count allows it (a 64-bit one is a hundred instructions)
    const int64_t tok = !live ? 0 : a.n_blocks <= 0xffffffffll ? (int64_t)((uint32_t)b / (uint32_t)per_tok) : b / per_tok;
    const int in_tok = live ? (int)(b - tok * per_tok) : 0, head = (int)((unsigned)in_tok / (unsigned)a.nb), blk = in_tok - head * a.nb;
    int64_t slot = live ? a.slots[tok] : -1;
    if (slot < -1 || (slot >= 0 && (slot >> a.pool.page_log2) >= a.pool.n_pages)) {
        atomicOr(a.status, STATUS_BAD_PAGE);
        slot = -1;
    }
    float k[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    int64_t at = 0;
    if (slot >= 0) {
        load8<BF16>(a.k, tok * a.k_stride + in_tok * 32 + 8 * e, a.k_vec, k);
        load8<BF16>(a.v, tok * a.v_stride + in_tok * 32 + 8 * e, a.v_vec, v);
        at = pool_row(a.pool, slot >> a.pool.page_log2, head, (int)(slot & ((1 << a.pool.page_log2) - 1))) + blk * Fmt<T>::BB;
    }
    append_block<T>(k, slot >= 0 ? a.K + at : nullptr, e);
    append_block<T>(v, slot >= 0 ? a.V + at : nullptr, e);
}

template <int T>
static cudaError_t append_t(const AppendArgs& a, bool bf16, cudaStream_t s) {
    const int64_t grid = (a.n_blocks * 4 + kAppendThreads - 1) / kAppendThreads;
    if (bf16) append_kernel<T, true><<<(unsigned)grid, kAppendThreads, 0, s>>>(a);
    else append_kernel<T, false><<<(unsigned)grid, kAppendThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// -------------------------------------------------------------- compact --
// One CTA per (request, pool, kv head): the accepted rows go through shared
// memory (at most 64 rows of 272 bytes), so that all are read before any is
// written.  Rows are copied in 2-byte units (a row is 2-byte aligned).  2.8 us
// for one request, 5.6 us for 61 of up to 29 rows: latency.
constexpr int kCompactThreads = 128;
constexpr int kTreeMax = 64;

struct CompactArgs {
    uint8_t* pool[2];
    Pool geo;
    const int32_t* table;
    int64_t table_stride;
    const int32_t *base, *path;
    int64_t path_stride;
    const int32_t* n_path;
    unsigned* status;
};

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactArgs a) {
    __shared__ uint16_t buf[kTreeMax * 136];
    __shared__ int64_t src[kTreeMax], dst[kTreeMax];
    const int64_t r = blockIdx.x;
    const int head = blockIdx.y >> 1, tid = threadIdx.x;
    uint8_t* pool = a.pool[blockIdx.y & 1];
    const int n = (int)min((int64_t)min(a.n_path[r], kTreeMax), a.path_stride);
    if (tid < n) {
        const int j = a.path[r * a.path_stride + tid];
        const int64_t base = a.base[r];
        src[tid] = -1;
        if (j != tid) {
            if (j >= 0 && j < kTreeMax && base >= 0) {
                const int32_t* tab = a.table + r * a.table_stride;
                const int64_t from = base + j, to = base + tid, mask = (1 << a.geo.page_log2) - 1;
                const int pf = page_of(a.geo, tab, a.table_stride, from, a.status);
                const int pt = page_of(a.geo, tab, a.table_stride, to, a.status);
                if (pf >= 0 && pt >= 0) {
                    src[tid] = pool_row(a.geo, pf, head, (int)(from & mask));
                    dst[tid] = pool_row(a.geo, pt, head, (int)(to & mask));
                }
            } else {
                atomicOr(a.status, STATUS_BAD_PAGE);
            }
        }
    }
    __syncthreads();
    const int units = a.geo.row_bytes / 2;
    for (int i = tid; i < n * units; i += kCompactThreads) {
        const int row = i / units, u = i - row * units;
        if (src[row] >= 0) buf[i] = reinterpret_cast<const uint16_t*>(pool + src[row])[u];
    }
    __syncthreads();
    for (int i = tid; i < n * units; i += kCompactThreads) {
        const int row = i / units, u = i - row * units;
        if (src[row] >= 0) reinterpret_cast<uint16_t*>(pool + dst[row])[u] = buf[i];
    }
}

}  // namespace kv

cudaError_t launch_kv_plan(const int32_t* have, const int32_t* start, const int32_t* want, int n_req, int page_log2,
                           int32_t* table, int64_t table_stride, int32_t* free_pages, int64_t free_cap,
                           const int32_t* n_free, int32_t* n_free_out, int32_t* granted, int32_t* cu, int64_t* slots,
                           int32_t* pos, int32_t* req, int64_t cap, int sms, cudaStream_t s) {
    const kv::PlanArgs a{have, start, want, n_req, page_log2, table, table_stride, free_pages, free_cap, n_free,
                         n_free_out, granted, cu, slots, pos, req, cap};
    // The limit is the kernel's, not the launch's: always the largest call's, so that another thread's smaller call
    // cannot lower it between these two lines.
    auto bytes = [](int n) { return 3 * (n + 1) * (int)sizeof(int); };
    const int smem = bytes(n_req);
    const cudaError_t e = cudaFuncSetAttribute(kv::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(QK_PLAN_MAX_REQ));
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>(std::max<int64_t>(1, (cap + kv::kTokensPerCta - 1) / kv::kTokensPerCta), sms);
    kv::plan_kernel<<<(unsigned)grid, kv::kPlanThreads, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(int type, const void* k, const void* v, bool bf16, int64_t n_tok, int64_t k_stride,
                             int64_t v_stride, int n_kv, int d, const int64_t* slots, uint8_t* K, uint8_t* V,
                             int64_t n_pages, int page_log2, int row_bytes, unsigned* status, cudaStream_t s) {
    const int es = bf16 ? 2 : 4;
    auto vec = [&](const void* p, int64_t stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0;
    };
    const int nb = d / 32;
    const kv::AppendArgs a{k, v, n_tok, k_stride, v_stride, slots, K, V, Pool{n_pages, page_log2, n_kv, row_bytes}, nb,
                           n_tok * n_kv * nb, vec(k, k_stride), vec(v, v_stride), status};
    switch (type) {
    case T_Q8_0: return kv::append_t<T_Q8_0>(a, bf16, s);
    case T_Q5_0: return kv::append_t<T_Q5_0>(a, bf16, s);
    case T_Q4_0: return kv::append_t<T_Q4_0>(a, bf16, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kv_compact(uint8_t* K, uint8_t* V, int64_t n_pages, int page_log2, int n_kv, int row_bytes,
                              const int32_t* table, int64_t table_stride, const int32_t* base, const int32_t* path,
                              int64_t path_stride, const int32_t* n_path, int64_t n_req, unsigned* status,
                              cudaStream_t s) {
    const kv::CompactArgs a{{K, V}, Pool{n_pages, page_log2, n_kv, row_bytes}, table, table_stride, base, path,
                            path_stride, n_path, status};
    kv::compact_kernel<<<dim3((unsigned)n_req, 2 * n_kv), kv::kCompactThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace qk
